// api.cu — the C ABI declared in include/lat_attn.h: argument validation, launch planning,
// tensor-map encoding and dispatch to the kernels.  No allocation, no global mutable state
// (the driver entry point for tensor-map encoding is resolved once and then read-only).
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <mutex>

#include "cache_kernels.h"
#include "kernels.h"
#include "lat_attn.h"
#include "lat_attn_testing.h"
#include "q8_block.cuh"

namespace {

bool supported_head_dim(int d) { return d == 64 || d == 80 || d == 128 || d == 256 || d == 512; }

// x / softcap for a score cap, kept where twice log2(e) times it is still a float: a cap so small
// that this matters takes every score but 0 to its ends, and 0 must not meet an infinity
float over_cap(float x, float softcap) { return fminf(fmaxf(x / softcap, -1e38f), 1e38f); }

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// 4-D bf16 map over (head-dim d, head, row, batch) with a [64, 1, box_rows, 1] box and
// 128-byte swizzle.  Columns past head_dim and rows past `rows` read as zero.
bool make_head_map(CUtensorMap *m, const void *base, int head_dim, int heads, int rows,
                   int batch, int64_t row_stride, int box_rows) {
    EncodeTiledFn fn = encode_tiled_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)head_dim, (cuuint64_t)heads, (cuuint64_t)rows,
                                (cuuint64_t)batch};
    const cuuint64_t strides[3] = {(cuuint64_t)head_dim * 2, (cuuint64_t)row_stride * 2,
                                   (cuuint64_t)row_stride * 2 * (cuuint64_t)rows};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)box_rows, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides,
              box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 4-D bf16 map over a KV cache: (head-dim d, KV head, row < rows, sequence) with the
// cache's own element strides, a [64, 1, box_rows, 1] box and 128-byte swizzle.
bool make_cache_map(CUtensorMap *m, const void *base, int head_dim, int heads, int rows,
                    int batch, int64_t row_stride, int64_t head_stride, int64_t seq_stride,
                    int box_rows,
                    CUtensorMapL2promotion promo = CU_TENSOR_MAP_L2_PROMOTION_L2_256B) {
    EncodeTiledFn fn = encode_tiled_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)head_dim, (cuuint64_t)heads, (cuuint64_t)rows,
                                (cuuint64_t)batch};
    const cuuint64_t strides[3] = {(cuuint64_t)head_stride * 2, (cuuint64_t)row_stride * 2,
                                   (cuuint64_t)seq_stride * 2};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)box_rows, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides,
              box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, promo,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 5-D bf16 map over the same tensor as make_cache_map, with the head dimension split into
// 64-column chunks: (d in chunk, row < rows, chunk, head, batch), 128-byte swizzle, box
// [64, box_rows, box_chunks, 1, 1].  One box lands as box_chunks consecutive
// [box_rows x 128 B] chunks: a whole multi-chunk tile in one copy.
bool make_chunked_map(CUtensorMap *m, const void *base, int head_dim, int heads, int rows,
                      int batch, int64_t row_stride, int64_t head_stride, int64_t seq_stride,
                      int box_rows, int box_chunks,
                      CUtensorMapL2promotion promo = CU_TENSOR_MAP_L2_PROMOTION_L2_128B) {
    EncodeTiledFn fn = encode_tiled_fn();
    if (fn == nullptr || head_dim % 64 != 0) return false;
    const cuuint64_t dims[5] = {64, (cuuint64_t)rows, (cuuint64_t)(head_dim / 64),
                                (cuuint64_t)heads, (cuuint64_t)batch};
    const cuuint64_t strides[4] = {(cuuint64_t)row_stride * 2, 128, (cuuint64_t)head_stride * 2,
                                   (cuuint64_t)seq_stride * 2};
    const cuuint32_t box[5] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_chunks, 1, 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(base), dims, strides,
              box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, promo,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 3-D bf16 map over decode queries: (head-dim d, query head, sequence), 8-head boxes
bool make_query_map(CUtensorMap *m, const void *base, int head_dim, int heads, int batch,
                    int64_t row_stride) {
    EncodeTiledFn fn = encode_tiled_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)heads, (cuuint64_t)batch};
    const cuuint64_t strides[2] = {(cuuint64_t)head_dim * 2, (cuuint64_t)row_stride * 2};
    const cuuint32_t box[3] = {64, 8, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides,
              box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 3-D bf16 map over a prefill output: (column < heads * head_dim, row < rows, batch) with
// 32-row boxes of box_cols columns, swizzled to the box's row width (128 or 64 bytes).
// Stores clip at the row extent, so rows past a sequence's end are never written.
bool make_out_map(CUtensorMap *m, void *base, int head_dim, int heads, int rows, int batch,
                  int64_t row_stride, int box_cols) {
    EncodeTiledFn fn = encode_tiled_fn();
    if (fn == nullptr || (box_cols != 64 && box_cols != 32)) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)heads * (cuuint64_t)head_dim, (cuuint64_t)rows,
                                (cuuint64_t)batch};
    const cuuint64_t strides[2] = {(cuuint64_t)row_stride * 2,
                                   (cuuint64_t)row_stride * 2 * (cuuint64_t)rows};
    const cuuint32_t box[3] = {(cuuint32_t)box_cols, 32, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE,
              box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int current_sm_count(int *out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    return cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr uint64_t kDefaultTimeoutNs = 4000000000ull;  // 4 s per CTA

// Where K and V element (b, j, hk, d) live: base + b*seq + j*row + hk*head + d (elements).
struct KvStrides {
    int64_t k_row, k_head, k_seq, v_row, v_head, v_seq;
};

lat_status prefill_impl(lat_dtype dt, const void *q, int64_t q_rs, const void *k, const void *v,
                        const KvStrides &kv, void *out, int64_t out_rs, float *lse, int batch,
                        int seq_len, int kv_len, int n_heads, int n_kv_heads, int head_dim,
                        int causal, int window, float scale, float softcap, int32_t *status,
                        void *stream, uint64_t timeout_ns, int skip_kv_load) {
    if (dt != LAT_F32 && dt != LAT_BF16) return LAT_ERR_INVALID_ARG;
    if (!(softcap >= 0.f) || !isfinite(softcap)) return LAT_ERR_INVALID_ARG;
    if (batch < 0 || seq_len < 0 || kv_len < seq_len || n_heads <= 0 || n_kv_heads <= 0 ||
        n_heads % n_kv_heads != 0)
        return LAT_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim)) return LAT_ERR_UNSUPPORTED;
    if (!isfinite(scale)) return LAT_ERR_INVALID_ARG;
    if (batch == 0 || seq_len == 0) return LAT_OK;
    if (!q || !k || !v || !out) return LAT_ERR_INVALID_ARG;
    if (q_rs < (int64_t)n_heads * head_dim || out_rs < (int64_t)n_heads * head_dim ||
        kv.k_row <= 0 || kv.k_head <= 0 || kv.k_seq <= 0 || kv.v_row <= 0 || kv.v_head <= 0 ||
        kv.v_seq <= 0)
        return LAT_ERR_INVALID_ARG;
    if (batch > 65535 || (seq_len + 127) / 128 > 65535) return LAT_ERR_UNSUPPORTED;
    if (window < 0) window = 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);

    if (dt == LAT_F32) {
        lat::RowAttnArgs a{};
        a.q = static_cast<const float *>(q);
        a.q_rs = q_rs;
        a.k = static_cast<const float *>(k);
        a.v = static_cast<const float *>(v);
        a.k_seq = kv.k_seq;
        a.k_row = kv.k_row;
        a.k_head = kv.k_head;
        a.v_seq = kv.v_seq;
        a.v_row = kv.v_row;
        a.v_head = kv.v_head;
        a.out = static_cast<float *>(out);
        a.out_rs = out_rs;
        a.lse = lse;
        a.batch = batch;
        a.seq_len = seq_len;
        a.kv_len = kv_len;
        a.n_heads = n_heads;
        a.n_kv_heads = n_kv_heads;
        a.head_dim = head_dim;
        a.causal = causal != 0;
        a.window = window;
        a.scale = scale;
        a.softcap = softcap;
        a.kv_lens = nullptr;
        a.max_kv_len = kv_len;
        a.status = status;
        return lat::launch_row_attention_f32(a, s) == cudaSuccess ? LAT_OK : LAT_ERR_CUDA;
    }

    // bf16: tensor-memory-access reads need 16-byte aligned bases and row strides
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || q_rs % 8 ||
        out_rs % 8 || kv.k_row % 8 || kv.k_head % 8 || kv.k_seq % 8 || kv.v_row % 8 ||
        kv.v_head % 8 || kv.v_seq % 8)
        return LAT_ERR_INVALID_ARG;
    if (lat::prefill_tc_items(batch, n_heads, head_dim, seq_len) > lat::kPrefillMaxItems)
        return LAT_ERR_UNSUPPORTED;
    lat::PrefillTcArgs a{};
    a.wide = lat::prefill_tc_wide(head_dim, seq_len, kv_len, causal, window) ? 1 : 0;
    a.pair = lat::prefill_tc_pair(head_dim, n_heads, n_kv_heads) ? 1 : 0;
    const int k_box = lat::prefill_tc_box_rows(head_dim, a.wide != 0, a.pair != 0, false);
    const int v_box = lat::prefill_tc_box_rows(head_dim, a.wide != 0, a.pair != 0, true);
    // K/V maps span exactly kv_len rows per sequence: rows past it read as zeros, so cache
    // slots beyond the visible keys (which may hold anything) never reach the MMA.  Head
    // dims that are whole 64-column chunks move each tile in one copy (chunked maps: Q all
    // chunks of 128 rows, K all chunks of its rows, V the chunks of this CTA's columns).
    a.chunked = lat::prefill_tc_chunked(head_dim, a.pair != 0) ? 1 : 0;
    if (a.chunked) {
        const int v_chunks = lat::prefill_tc_v_chunks(head_dim, a.pair != 0);
        if (!make_chunked_map(&a.tm_q, q, head_dim, n_heads, seq_len, batch, q_rs, head_dim,
                              (int64_t)seq_len * q_rs, 128, head_dim / 64) ||
            !make_chunked_map(&a.tm_k, k, head_dim, n_kv_heads, kv_len, batch, kv.k_row,
                              kv.k_head, kv.k_seq, k_box, head_dim / 64) ||
            !make_chunked_map(&a.tm_v, v, head_dim, n_kv_heads, kv_len, batch, kv.v_row,
                              kv.v_head, kv.v_seq, v_box, v_chunks))
            return LAT_ERR_CUDA;
    } else if (!make_head_map(&a.tm_q, q, head_dim, n_heads, seq_len, batch, q_rs, 128) ||
        !make_cache_map(&a.tm_k, k, head_dim, n_kv_heads, kv_len, batch, kv.k_row, kv.k_head,
                        kv.k_seq, k_box, CU_TENSOR_MAP_L2_PROMOTION_L2_128B) ||
        !make_cache_map(&a.tm_v, v, head_dim, n_kv_heads, kv_len, batch, kv.v_row, kv.v_head,
                        kv.v_seq, v_box, CU_TENSOR_MAP_L2_PROMOTION_L2_128B))
        return LAT_ERR_CUDA;
    const int out_box = lat::prefill_tc_out_box_cols(head_dim, a.pair != 0);
    if (out_box > 0 &&
        !make_out_map(&a.tm_out, out, head_dim, n_heads, seq_len, batch, out_rs, out_box))
        return LAT_ERR_CUDA;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.out_rs = out_rs;
    a.out_v8 = reinterpret_cast<uintptr_t>(out) % 32 == 0 && out_rs % 16 == 0;
    a.lse = lse;
    a.batch = batch;
    a.seq_len = seq_len;
    a.kv_len = kv_len;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.causal = causal != 0;
    a.window = window;
    a.scale_log2 = scale * kLog2e;
    a.cap_log2 = softcap > 0.f ? softcap * kLog2e : 0.f;
    a.raw_over_cap = softcap > 0.f ? over_cap(scale, softcap) : 0.f;
    a.status = status;
    a.timeout_ns = timeout_ns;
    a.test_skip_kv_load = skip_kv_load;
    int sms = 0;
    if (!current_sm_count(&sms)) return LAT_ERR_CUDA;
    return lat::launch_prefill_tc(a, sms, s) == cudaSuccess ? LAT_OK : LAT_ERR_CUDA;
}

}  // namespace

extern "C" {

const char *lat_status_string(lat_status st) {
    switch (st) {
        case LAT_OK: return "LAT_OK";
        case LAT_ERR_INVALID_ARG: return "LAT_ERR_INVALID_ARG";
        case LAT_ERR_UNSUPPORTED: return "LAT_ERR_UNSUPPORTED";
        case LAT_ERR_WORKSPACE: return "LAT_ERR_WORKSPACE";
        case LAT_ERR_CUDA: return "LAT_ERR_CUDA";
        case LAT_ERR_BOUNDS: return "LAT_ERR_BOUNDS";
        case LAT_ERR_TIMEOUT: return "LAT_ERR_TIMEOUT";
    }
    return "LAT_ERR_UNKNOWN";
}

lat_status lat_attn_prefill(lat_dtype dt, const void *q, int64_t q_rs, const void *k,
                            int64_t k_rs, const void *v, int64_t v_rs, void *out,
                            int64_t out_rs, float *lse, int batch, int seq_len, int kv_len,
                            int n_heads, int n_kv_heads, int head_dim, int causal, int window,
                            float scale, int32_t *status, void *stream) {
    if (k_rs < (int64_t)n_kv_heads * head_dim || v_rs < (int64_t)n_kv_heads * head_dim)
        return LAT_ERR_INVALID_ARG;
    const KvStrides kv{k_rs, head_dim, (int64_t)kv_len * k_rs, v_rs, head_dim, (int64_t)kv_len * v_rs};
    return prefill_impl(dt, q, q_rs, k, v, kv, out, out_rs, lse, batch, seq_len, kv_len, n_heads,
                        n_kv_heads, head_dim, causal, window, scale, 0.f, status, stream,
                        kDefaultTimeoutNs, 0);
}

lat_status lat_attn_prefill_softcap(lat_dtype dt, const void *q, int64_t q_rs, const void *k,
                                    int64_t k_rs, const void *v, int64_t v_rs, void *out,
                                    int64_t out_rs, float *lse, int batch, int seq_len,
                                    int kv_len, int n_heads, int n_kv_heads, int head_dim,
                                    int causal, int window, float scale, float softcap,
                                    int32_t *status, void *stream) {
    if (k_rs < (int64_t)n_kv_heads * head_dim || v_rs < (int64_t)n_kv_heads * head_dim)
        return LAT_ERR_INVALID_ARG;
    const KvStrides kv{k_rs, head_dim, (int64_t)kv_len * k_rs, v_rs, head_dim, (int64_t)kv_len * v_rs};
    return prefill_impl(dt, q, q_rs, k, v, kv, out, out_rs, lse, batch, seq_len, kv_len, n_heads,
                        n_kv_heads, head_dim, causal, window, scale, softcap, status, stream,
                        kDefaultTimeoutNs, 0);
}

lat_status lat_attn_prefill_cached(lat_dtype dt, const void *q, int64_t q_rs,
                                   const void *k_cache, const void *v_cache, int64_t cache_rs,
                                   int64_t cache_head_stride, int64_t cache_seq_stride,
                                   void *out, int64_t out_rs, float *lse, int batch,
                                   int seq_len, int kv_len, int n_heads, int n_kv_heads,
                                   int head_dim, int causal, int window, float scale,
                                   int32_t *status, void *stream) {
    const KvStrides kv{cache_rs, cache_head_stride, cache_seq_stride,
                       cache_rs, cache_head_stride, cache_seq_stride};
    return prefill_impl(dt, q, q_rs, k_cache, v_cache, kv, out, out_rs, lse, batch, seq_len,
                        kv_len, n_heads, n_kv_heads, head_dim, causal, window, scale, 0.f, status,
                        stream, kDefaultTimeoutNs, 0);
}

lat_status lat_test_prefill_timeout(const void *q, int64_t q_rs, const void *k, int64_t k_rs,
                                    const void *v, int64_t v_rs, void *out, int64_t out_rs,
                                    int batch, int seq_len, int n_heads, int n_kv_heads,
                                    int head_dim, uint64_t timeout_ns, int32_t *status,
                                    void *stream) {
    const KvStrides kv{k_rs, head_dim, (int64_t)seq_len * k_rs, v_rs, head_dim,
                       (int64_t)seq_len * v_rs};
    return prefill_impl(LAT_BF16, q, q_rs, k, v, kv, out, out_rs, nullptr, batch, seq_len,
                        seq_len, n_heads, n_kv_heads, head_dim, 1, 0, 0.125f, 0.f, status, stream,
                        timeout_ns, 1);
}

size_t lat_attn_decode_workspace_size(lat_dtype dt, int batch, int n_heads, int n_kv_heads,
                                      int head_dim, int max_kv_len) {
    if (dt == LAT_F32) return 0;
    if (dt != LAT_BF16 || batch < 0 || n_heads <= 0 || n_kv_heads <= 0 ||
        n_heads % n_kv_heads != 0 || !supported_head_dim(head_dim) || max_kv_len < 0)
        return 0;
    int sms = 0;
    if (!current_sm_count(&sms)) return 0;
    lat::DecodePlan plan;
    if (!lat::plan_decode_bf16(batch, n_heads, n_kv_heads, head_dim, max_kv_len, 0, sms, &plan))
        return 0;
    return plan.total_bytes;
}

}  // extern "C"

namespace {

lat_status decode_impl(lat_dtype dt, const void *q, int64_t q_rs, const void *k_cache,
                       const void *v_cache, int64_t cache_rs, int64_t cache_head_stride,
                       int64_t cache_seq_stride, const int32_t *kv_lens, int max_kv_len,
                       void *out, int64_t out_rs, float *lse, int batch, int n_heads,
                       int n_kv_heads, int head_dim, int window, float scale, float softcap,
                       int ring, void *workspace, size_t workspace_bytes, int32_t *status,
                       void *stream, uint64_t timeout_ns, int skip_load,
                       const int32_t *blocks = nullptr, int n_sel = 0, int block_size = 0) {
    if (dt != LAT_F32 && dt != LAT_BF16) return LAT_ERR_INVALID_ARG;
    if (!(softcap >= 0.f) || !isfinite(softcap)) return LAT_ERR_INVALID_ARG;
    // a ring cache keeps only the last `ring` positions: the window must fit in it
    if (ring < 0 || (ring > 0 && (window <= 0 || window > ring))) return LAT_ERR_INVALID_ARG;
    if (batch < 0 || max_kv_len < 0 || n_heads <= 0 || n_kv_heads <= 0 ||
        n_heads % n_kv_heads != 0)
        return LAT_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim)) return LAT_ERR_UNSUPPORTED;
    if (!isfinite(scale)) return LAT_ERR_INVALID_ARG;
    if (batch == 0) return LAT_OK;
    if (!q || !k_cache || !v_cache || !kv_lens || !out) return LAT_ERR_INVALID_ARG;
    if (q_rs < (int64_t)n_heads * head_dim || out_rs < (int64_t)n_heads * head_dim ||
        cache_rs <= 0 || cache_head_stride <= 0 || cache_seq_stride <= 0)
        return LAT_ERR_INVALID_ARG;
    if (batch > 65535) return LAT_ERR_UNSUPPORTED;
    if (window < 0) window = 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);

    if (dt == LAT_F32) {
        lat::RowAttnArgs a{};
        a.q = static_cast<const float *>(q);
        a.q_rs = q_rs;
        a.k = static_cast<const float *>(k_cache);
        a.v = static_cast<const float *>(v_cache);
        a.k_seq = a.v_seq = cache_seq_stride;
        a.k_row = a.v_row = cache_rs;
        a.k_head = a.v_head = cache_head_stride;
        a.out = static_cast<float *>(out);
        a.out_rs = out_rs;
        a.lse = lse;
        a.batch = batch;
        a.seq_len = 1;
        a.kv_len = 0;
        a.n_heads = n_heads;
        a.n_kv_heads = n_kv_heads;
        a.head_dim = head_dim;
        a.causal = 1;
        a.window = window;
        a.scale = scale;
        a.softcap = softcap;
        a.kv_lens = kv_lens;
        a.max_kv_len = max_kv_len;
        a.ring = ring;
        a.status = status;
        return lat::launch_row_attention_f32(a, s) == cudaSuccess ? LAT_OK : LAT_ERR_CUDA;
    }

    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
        q_rs % 8 || cache_rs % 8 || cache_head_stride % 8 || cache_seq_stride % 8 || out_rs % 8)
        return LAT_ERR_INVALID_ARG;
    if (lat::decode_bf16_units(batch, n_heads, n_kv_heads) >= lat::kDecodeMaxUnits)
        return LAT_ERR_UNSUPPORTED;
    int sms = 0;
    if (!current_sm_count(&sms)) return LAT_ERR_CUDA;
    // rows per sequence: the ring, or every position up to max_kv_len; the scratch layout
    // is sized by the same count (a ring's visible keys never exceed it)
    const int rows = ring > 0 ? ring : max_kv_len;
    // (over chosen blocks the stream is as long as the list at most)
    lat::DecodePlan plan;
    if (!(blocks != nullptr
              ? lat::plan_decode_blocks_bf16(batch, n_heads, n_kv_heads, head_dim, n_sel * block_size, sms, &plan)
              : lat::plan_decode_bf16(batch, n_heads, n_kv_heads, head_dim, rows, window, sms, &plan)))
        return LAT_ERR_UNSUPPORTED;
    if (workspace == nullptr || workspace_bytes < plan.total_bytes ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return LAT_ERR_WORKSPACE;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    lat::DecodeBlocksArgs a{};  // the dense decode's arguments are its first part
    if (max_kv_len > 0) {
        const int box = lat::decode_bf16_tile_keys(head_dim);
        // head dims of up to four whole 64-column chunks take each K (or V) tile in one
        // copy (at head_dim 512, eight 32-row chunks per copy measured 2.4 % slower than
        // eight copies)
        a.chunked = head_dim % 64 == 0 && head_dim <= 256 ? 1 : 0;
        const bool maps_ok =
            a.chunked
                ? make_chunked_map(&a.tm_k, k_cache, head_dim, n_kv_heads, rows, batch, cache_rs,
                                   cache_head_stride, cache_seq_stride, box, head_dim / 64,
                                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B) &&
                      make_chunked_map(&a.tm_v, v_cache, head_dim, n_kv_heads, rows, batch,
                                       cache_rs, cache_head_stride, cache_seq_stride, box,
                                       head_dim / 64, CU_TENSOR_MAP_L2_PROMOTION_L2_256B)
                : make_cache_map(&a.tm_k, k_cache, head_dim, n_kv_heads, rows, batch, cache_rs,
                                 cache_head_stride, cache_seq_stride, box) &&
                      make_cache_map(&a.tm_v, v_cache, head_dim, n_kv_heads, rows, batch,
                                     cache_rs, cache_head_stride, cache_seq_stride, box);
        const bool partial_ok =
            make_cache_map(&a.tm_k16, k_cache, head_dim, n_kv_heads, rows, batch, cache_rs,
                           cache_head_stride, cache_seq_stride, 16) &&
            make_cache_map(&a.tm_v16, v_cache, head_dim, n_kv_heads, rows, batch, cache_rs,
                           cache_head_stride, cache_seq_stride, 16);
        if (!maps_ok || !partial_ok ||
            !make_query_map(&a.tm_q, q, head_dim, n_heads, batch, q_rs))
            return LAT_ERR_CUDA;
    }
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.q_rs = q_rs;
    a.k_cache = static_cast<const __nv_bfloat16 *>(k_cache);
    a.v_cache = static_cast<const __nv_bfloat16 *>(v_cache);
    a.cache_rs = cache_rs;
    a.cache_head = cache_head_stride;
    a.cache_seq = cache_seq_stride;
    a.kv_lens = kv_lens;
    a.max_kv_len = max_kv_len;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.out_rs = out_rs;
    a.lse = lse;
    a.batch = batch;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.window = window;
    a.ring = ring;
    a.blocks = blocks;
    a.n_sel = n_sel;
    a.block_size = block_size;
    a.scale_log2 = scale * kLog2e;
    a.cap_log2 = softcap > 0.f ? softcap * kLog2e : 0.f;
    a.raw_over_cap = softcap > 0.f ? over_cap(scale, softcap) : 0.f;
    a.part_o = reinterpret_cast<float *>(ws);
    a.part_lse = reinterpret_cast<float *>(ws + plan.part_o_bytes);
    a.counters = reinterpret_cast<int32_t *>(ws + plan.part_o_bytes + plan.part_lse_bytes);
    a.max_splits = plan.max_splits;
    a.min_seg = plan.min_seg;
    a.defer_merge = plan.defer_merge;
    a.piece_count = a.counters;  // the same scratch region, used one way or the other
    a.timeout_ns = timeout_ns;
    a.test_skip_load = skip_load;
    a.status = status;
    return (blocks != nullptr ? lat::launch_decode_blocks_bf16(a, plan.grid, s)
                              : lat::launch_decode_bf16(a, plan.grid, s)) == cudaSuccess
               ? LAT_OK
               : LAT_ERR_CUDA;
}

}  // namespace

extern "C" {

lat_status lat_attn_decode(lat_dtype dt, const void *q, int64_t q_rs, const void *k_cache,
                           const void *v_cache, int64_t cache_rs, int64_t cache_head_stride,
                           int64_t cache_seq_stride, const int32_t *kv_lens, int max_kv_len,
                           void *out, int64_t out_rs, float *lse, int batch, int n_heads,
                           int n_kv_heads, int head_dim, int window, float scale,
                           void *workspace, size_t workspace_bytes, int32_t *status,
                           void *stream) {
    return decode_impl(dt, q, q_rs, k_cache, v_cache, cache_rs, cache_head_stride,
                       cache_seq_stride, kv_lens, max_kv_len, out, out_rs, lse, batch, n_heads,
                       n_kv_heads, head_dim, window, scale, 0.f, 0, workspace,
                       workspace_bytes, status, stream,
                       kDefaultTimeoutNs, 0);
}

lat_status lat_attn_decode_ring(lat_dtype dt, const void *q, int64_t q_rs, const void *k_cache,
                                const void *v_cache, int64_t cache_rs, int64_t cache_head_stride,
                                int64_t cache_seq_stride, int ring_capacity,
                                const int32_t *kv_lens, int max_kv_len, void *out,
                                int64_t out_rs, float *lse, int batch, int n_heads,
                                int n_kv_heads, int head_dim, int window, float scale,
                                void *workspace, size_t workspace_bytes, int32_t *status,
                                void *stream) {
    if (ring_capacity <= 0) return LAT_ERR_INVALID_ARG;
    return decode_impl(dt, q, q_rs, k_cache, v_cache, cache_rs, cache_head_stride,
                       cache_seq_stride, kv_lens, max_kv_len, out, out_rs, lse, batch, n_heads,
                       n_kv_heads, head_dim, window, scale, 0.f, ring_capacity, workspace,
                       workspace_bytes, status, stream,
                       kDefaultTimeoutNs, 0);
}

lat_status lat_attn_decode_softcap(lat_dtype dt, const void *q, int64_t q_rs,
                                   const void *k_cache, const void *v_cache, int64_t cache_rs,
                                   int64_t cache_head_stride, int64_t cache_seq_stride,
                                   const int32_t *kv_lens, int max_kv_len, void *out,
                                   int64_t out_rs, float *lse, int batch, int n_heads,
                                   int n_kv_heads, int head_dim, int window, float scale,
                                   float softcap, void *workspace, size_t workspace_bytes,
                                   int32_t *status, void *stream) {
    return decode_impl(dt, q, q_rs, k_cache, v_cache, cache_rs, cache_head_stride,
                       cache_seq_stride, kv_lens, max_kv_len, out, out_rs, lse, batch, n_heads,
                       n_kv_heads, head_dim, window, scale, softcap, 0, workspace,
                       workspace_bytes, status, stream,
                       kDefaultTimeoutNs, 0);
}

lat_status lat_test_decode_timeout(const void *q, int64_t q_rs, const void *k_cache,
                                   const void *v_cache, int64_t cache_rs,
                                   int64_t cache_head_stride, int64_t cache_seq_stride,
                                   const int32_t *kv_lens, int max_kv_len, void *out,
                                   int64_t out_rs, int batch, int n_heads, int n_kv_heads,
                                   int head_dim, void *workspace, size_t workspace_bytes,
                                   uint64_t timeout_ns, int32_t *status, void *stream) {
    return decode_impl(LAT_BF16, q, q_rs, k_cache, v_cache, cache_rs, cache_head_stride,
                       cache_seq_stride, kv_lens, max_kv_len, out, out_rs, nullptr, batch,
                       n_heads, n_kv_heads, head_dim, 0, 0.125f, 0.f, 0, workspace,
                       workspace_bytes, status, stream, timeout_ns, 1);
}

lat_status lat_test_capped_scores(const float *raw, int64_t n, float scale, float softcap,
                                  float *out, void *stream) {
    if (n < 0 || !(softcap > 0.f) || !isfinite(scale)) return LAT_ERR_INVALID_ARG;
    if (n == 0) return LAT_OK;
    if (raw == nullptr || out == nullptr) return LAT_ERR_INVALID_ARG;
    // the same two factors the attention entry points hand their kernels
    return lat::launch_capped_scores(raw, n, over_cap(scale, softcap), softcap * kLog2e, out,
                                     static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? LAT_OK
               : LAT_ERR_CUDA;
}

}  // extern "C"

namespace {

lat_status append_impl(lat_dtype dt, void *k_cache, void *v_cache, int64_t cache_rs,
                       int64_t cache_head_stride, int64_t cache_seq_stride, int capacity,
                       const void *k_new, const void *v_new, int64_t new_rs, const int32_t *pos,
                       int n_new, int batch, int n_kv_heads, int head_dim, int ring,
                       int32_t *status, void *stream) {
    if (dt != LAT_F32 && dt != LAT_BF16) return LAT_ERR_INVALID_ARG;
    if (batch < 0 || n_new < 0 || capacity < 0 || n_kv_heads <= 0) return LAT_ERR_INVALID_ARG;
    if (ring > 0 && n_new > ring) return LAT_ERR_INVALID_ARG;  // rows would overwrite each other
    if (!supported_head_dim(head_dim)) return LAT_ERR_UNSUPPORTED;
    if (batch == 0 || n_new == 0) return LAT_OK;
    if (!k_cache || !v_cache || !k_new || !v_new || !pos) return LAT_ERR_INVALID_ARG;
    if (cache_rs <= 0 || cache_head_stride <= 0 || cache_seq_stride <= 0 ||
        new_rs < (int64_t)n_kv_heads * head_dim)
        return LAT_ERR_INVALID_ARG;
    lat::AppendArgs a{};
    a.k_cache = static_cast<char *>(k_cache);
    a.v_cache = static_cast<char *>(v_cache);
    a.k_new = static_cast<const char *>(k_new);
    a.v_new = static_cast<const char *>(v_new);
    a.cache_rs = cache_rs;
    a.cache_head = cache_head_stride;
    a.cache_seq = cache_seq_stride;
    a.new_rs = new_rs;
    a.pos = pos;
    a.capacity = capacity;
    a.n_new = n_new;
    a.batch = batch;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.elem_bytes = dt == LAT_F32 ? 4 : 2;
    a.ring = ring;
    a.status = status;
    return lat::launch_kv_append(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? LAT_OK
               : LAT_ERR_CUDA;
}

}  // namespace

extern "C" {

lat_status lat_kv_append(lat_dtype dt, void *k_cache, void *v_cache, int64_t cache_rs,
                         int64_t cache_head_stride, int64_t cache_seq_stride, int capacity,
                         const void *k_new, const void *v_new, int64_t new_rs,
                         const int32_t *pos, int n_new, int batch, int n_kv_heads,
                         int head_dim, int32_t *status, void *stream) {
    return append_impl(dt, k_cache, v_cache, cache_rs, cache_head_stride, cache_seq_stride,
                       capacity, k_new, v_new, new_rs, pos, n_new, batch, n_kv_heads, head_dim,
                       0, status, stream);
}

lat_status lat_qkv_norm_rope_append(lat_dtype dt, const void *qkv, int64_t qkv_rs,
                                    const void *q_norm_w, const void *k_norm_w, float eps,
                                    double rope_base, int v_unit_norm, void *q_out,
                                    int64_t q_out_rs, void *k_cache, void *v_cache,
                                    int64_t cache_rs, int64_t cache_head_stride,
                                    int64_t cache_seq_stride, int capacity, const int32_t *pos,
                                    int n_new, int batch, int n_heads, int n_kv_heads,
                                    int head_dim, int32_t *status, void *stream) {
    if (dt != LAT_F32 && dt != LAT_BF16) return LAT_ERR_INVALID_ARG;
    if (batch < 0 || n_new < 0 || capacity < 0 || n_heads <= 0 || n_kv_heads <= 0 ||
        n_heads % n_kv_heads != 0)
        return LAT_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim)) return LAT_ERR_UNSUPPORTED;
    if (!(eps >= 0.f) || !isfinite(eps) || !(rope_base > 1.0) || !isfinite(rope_base))
        return LAT_ERR_INVALID_ARG;
    if (batch == 0 || n_new == 0) return LAT_OK;
    if (!qkv || !q_out || !k_cache || !v_cache || !pos) return LAT_ERR_INVALID_ARG;
    if (qkv_rs < (int64_t)(n_heads + 2 * n_kv_heads) * head_dim ||
        q_out_rs < (int64_t)n_heads * head_dim || cache_rs <= 0 || cache_head_stride <= 0 ||
        cache_seq_stride <= 0)
        return LAT_ERR_INVALID_ARG;
    lat::ProducerArgs a{};
    a.qkv = qkv;
    a.qkv_rs = qkv_rs;
    a.q_w = q_norm_w;
    a.k_w = k_norm_w;
    a.eps = eps;
    a.v_unit_norm = v_unit_norm != 0;
    a.q_out = q_out;
    a.q_out_rs = q_out_rs;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.cache_rs = cache_rs;
    a.cache_head = cache_head_stride;
    a.cache_seq = cache_seq_stride;
    a.capacity = capacity;
    a.pos = pos;
    a.n_new = n_new;
    a.batch = batch;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.status = status;
    for (int i = 0; i < head_dim / 2; ++i)  // the rotation frequencies, in double
        a.inv_freq[i] = pow(rope_base, -2.0 * i / head_dim);
    return lat::launch_qkv_producer(a, dt == LAT_BF16, reinterpret_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? LAT_OK
               : LAT_ERR_CUDA;
}

lat_status lat_kv_append_ring(lat_dtype dt, void *k_cache, void *v_cache, int64_t cache_rs,
                              int64_t cache_head_stride, int64_t cache_seq_stride,
                              int ring_capacity, const void *k_new, const void *v_new,
                              int64_t new_rs, const int32_t *pos, int n_new, int batch,
                              int n_kv_heads, int head_dim, int32_t *status, void *stream) {
    if (ring_capacity <= 0) return LAT_ERR_INVALID_ARG;
    return append_impl(dt, k_cache, v_cache, cache_rs, cache_head_stride, cache_seq_stride,
                       ring_capacity, k_new, v_new, new_rs, pos, n_new, batch, n_kv_heads,
                       head_dim, ring_capacity, status, stream);
}

}  // extern "C"

// ---------------------------------------------------------------- 4-bit KV cache

namespace {

// Map of a 4-bit cache in 32-bit words.  Rows of whole 128-byte pieces: 5-D, (word of the piece,
// row < rows, piece, KV head, sequence) with a [32, box_rows, pieces, 1, 1] box and the 128-byte
// swizzle; others 4-D, (word of the row, KV head, row, sequence) with a [row, 1, box_rows, 1] box.
// L2 fetches 64 bytes at a time: a row of a token-major cache lies apart from the next one of its
// head, and fetching 256 bytes about it cost 40 % (32 x 8192 keys, 8 KV heads of 128: 113 us, by
// 64 bytes 81).
bool make_q4_map(CUtensorMap *m, const void *base, int row_bytes, int heads, int rows, int batch,
                 int64_t row_stride, int64_t head_stride, int64_t seq_stride, int box_rows) {
    EncodeTiledFn fn = encode_tiled_fn();
    if (fn == nullptr) return false;
    const cuuint64_t w = (cuuint64_t)row_bytes / 4, h = (cuuint64_t)heads, n = (cuuint64_t)rows, b = (cuuint64_t)batch;
    const cuuint64_t rs = (cuuint64_t)row_stride, hs = (cuuint64_t)head_stride, ss = (cuuint64_t)seq_stride;
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    if (row_bytes % 128 == 0) {
        const cuuint64_t dims[5] = {32, n, w / 32, h, b}, strides[4] = {rs, 128, hs, ss};
        const cuuint32_t box[5] = {32, (cuuint32_t)box_rows, (cuuint32_t)w / 32, 1, 1};
        return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 5, const_cast<void *>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_64B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    }
    const cuuint64_t dims[4] = {w, h, n, b}, strides[3] = {hs, rs, ss};
    const cuuint32_t box[4] = {(cuuint32_t)w, 1, (cuuint32_t)box_rows, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_64B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// a query row's elements are counted in 32 bits by the decodes over reduced caches
bool query_row_ok(int n_heads, int head_dim) { return (int64_t)n_heads * head_dim <= 0x7fffffffLL; }

// a score cap whose products with log2(e) and 2 stay floats and whose reciprocal keeps its bits
float cap_in_range(float softcap) { return fminf(softcap, 1e36f); }

bool q4_strides_ok(int64_t row, int64_t head, int64_t seq) {
    return row > 0 && head > 0 && seq > 0 && row % 16 == 0 && head % 16 == 0 && seq % 16 == 0;
}

lat_status q4_store_impl(lat_dtype dt, void *cache, int64_t cache_rs, int64_t cache_head_stride,
                         int64_t cache_seq_stride, int capacity, const void *k, const void *v, void *k_out,
                         void *v_out, int64_t rs, const int32_t *pos, int n, int batch, int n_kv_heads,
                         int head_dim, bool expand, int32_t *status, void *stream) {
    if (dt != LAT_F32 && dt != LAT_BF16) return LAT_ERR_INVALID_ARG;
    if (batch < 0 || n < 0 || capacity < 0 || n_kv_heads <= 0) return LAT_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim)) return LAT_ERR_UNSUPPORTED;
    if (batch == 0 || n == 0) return LAT_OK;
    if (!cache || !pos || (expand ? (!k_out || !v_out) : (!k || !v))) return LAT_ERR_INVALID_ARG;
    if (!aligned16(cache) || !q4_strides_ok(cache_rs, cache_head_stride, cache_seq_stride) ||
        rs < (int64_t)n_kv_heads * head_dim)
        return LAT_ERR_INVALID_ARG;
    if ((int64_t)batch * n > 0x7fffffffLL / n_kv_heads) return LAT_ERR_UNSUPPORTED;
    lat::Q4StoreArgs a{};
    a.cache = static_cast<unsigned char *>(cache);
    a.cache_rs = cache_rs;
    a.cache_head = cache_head_stride;
    a.cache_seq = cache_seq_stride;
    a.k = k;
    a.v = v;
    a.k_out = k_out;
    a.v_out = v_out;
    a.rs = rs;
    const int64_t es = dt == LAT_BF16 ? 2 : 4;
    a.vec = rs * es % 16 == 0 && (expand ? aligned16(k_out) && aligned16(v_out) : aligned16(k) && aligned16(v));
    a.pos = pos;
    a.capacity = capacity;
    a.n = n;
    a.batch = batch;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.by_heads = lat::FastDiv((uint32_t)n_kv_heads);
    a.by_n = lat::FastDiv((uint32_t)n);
    a.status = status;
    return lat::launch_q4_store(a, dt == LAT_BF16, expand, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? LAT_OK
               : LAT_ERR_CUDA;
}

// what the decodes over packed caches have in common; `workspace` holds plan.total_bytes
void fill_split_args(lat::SplitDecodeArgs &a, const lat::SplitPlan &plan, const void *q, int64_t q_rs,
                     const int32_t *kv_lens, int max_kv_len, void *out, int64_t out_rs, float *lse, int batch,
                     int n_heads, int n_kv_heads, int head_dim, int window, float scale, float softcap,
                     void *workspace, int32_t *status, uint64_t timeout_ns, int skip_load) {
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    a.q = q;
    a.q_rs = q_rs;
    a.kv_lens = kv_lens;
    a.max_kv_len = max_kv_len;
    a.out = out;
    a.out_rs = out_rs;
    a.lse = lse;
    a.batch = batch;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.window = window < 0 ? 0 : window;
    a.scale_log2 = scale * kLog2e;
    softcap = cap_in_range(softcap);
    a.cap_log2 = softcap > 0.f ? softcap * kLog2e : 0.f;
    a.over_cap_log2 = softcap > 0.f ? over_cap(1.f, softcap * kLog2e) : 0.f;
    a.part_o = reinterpret_cast<float *>(ws);
    a.part_lse = reinterpret_cast<float *>(ws + plan.part_o_bytes);
    a.piece_count = a.counters = reinterpret_cast<int32_t *>(ws + plan.part_o_bytes + plan.part_lse_bytes);
    a.defer_join = plan.defer_join;
    a.max_splits = plan.max_splits;
    a.min_tiles = plan.min_tiles;
    a.whole = plan.whole;
    a.timeout_ns = timeout_ns;
    a.test_skip_load = skip_load;
    a.status = status;
}

lat_status q4_decode_impl(lat_dtype dt, const void *q, int64_t q_rs, const void *cache, int64_t cache_rs,
                          int64_t cache_head_stride, int64_t cache_seq_stride, const int32_t *kv_lens,
                          int max_kv_len, void *out, int64_t out_rs, float *lse, int batch, int n_heads,
                          int n_kv_heads, int head_dim, int window, float scale, float softcap,
                          void *workspace, size_t workspace_bytes, int32_t *status, void *stream,
                          uint64_t timeout_ns, int skip_load) {
    if (dt != LAT_F32 && dt != LAT_BF16) return LAT_ERR_INVALID_ARG;
    if (!(softcap >= 0.f) || !isfinite(softcap) || !isfinite(scale)) return LAT_ERR_INVALID_ARG;
    if (batch < 0 || max_kv_len < 0 || n_heads <= 0 || n_kv_heads <= 0 || n_heads % n_kv_heads != 0)
        return LAT_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim)) return LAT_ERR_UNSUPPORTED;
    if (batch == 0) return LAT_OK;
    if (!q || !cache || !kv_lens || !out) return LAT_ERR_INVALID_ARG;
    const int64_t per16 = dt == LAT_BF16 ? 8 : 4;  // elements in 16 bytes
    if (q_rs < (int64_t)n_heads * head_dim || out_rs < (int64_t)n_heads * head_dim || q_rs % per16 ||
        out_rs % per16 || !aligned16(q) || !aligned16(cache) || !aligned16(out) ||
        !q4_strides_ok(cache_rs, cache_head_stride, cache_seq_stride))
        return LAT_ERR_INVALID_ARG;
    if (batch > 65535 || !query_row_ok(n_heads, head_dim)) return LAT_ERR_UNSUPPORTED;
    int sms = 0;
    if (!current_sm_count(&sms)) return LAT_ERR_CUDA;
    lat::Q4Plan plan;
    if (!lat::plan_decode_q4(batch, n_heads, n_kv_heads, head_dim, dt == LAT_BF16, max_kv_len, sms, &plan))
        return LAT_ERR_UNSUPPORTED;
    if (workspace == nullptr || workspace_bytes < plan.total_bytes ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return LAT_ERR_WORKSPACE;
    lat::Q4DecodeArgs a{};
    if (max_kv_len > 0 &&
        !make_q4_map(&a.tm, cache, lat::q4_row_bytes(head_dim), n_kv_heads, max_kv_len, batch, cache_rs,
                     cache_head_stride, cache_seq_stride, plan.box_rows))
        return LAT_ERR_CUDA;
    fill_split_args(a, plan, q, q_rs, kv_lens, max_kv_len, out, out_rs, lse, batch, n_heads, n_kv_heads, head_dim,
                    window, scale, softcap, workspace, status, timeout_ns, skip_load);
    return lat::launch_decode_q4(a, dt == LAT_BF16, plan, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? LAT_OK
               : LAT_ERR_CUDA;
}

}  // namespace

extern "C" {

int lat_kv_q4_row_bytes(int head_dim) { return lat::q4_row_bytes(head_dim); }

lat_status lat_kv_append_q4(lat_dtype dt, void *cache, int64_t cache_rs, int64_t cache_head_stride,
                            int64_t cache_seq_stride, int capacity, const void *k_new, const void *v_new,
                            int64_t new_rs, const int32_t *pos, int n_new, int batch, int n_kv_heads,
                            int head_dim, int32_t *status, void *stream) {
    return q4_store_impl(dt, cache, cache_rs, cache_head_stride, cache_seq_stride, capacity, k_new, v_new, nullptr,
                         nullptr, new_rs, pos, n_new, batch, n_kv_heads, head_dim, false, status, stream);
}

lat_status lat_kv_expand_q4(lat_dtype dt, const void *cache, int64_t cache_rs, int64_t cache_head_stride,
                            int64_t cache_seq_stride, int capacity, void *k_out, void *v_out, int64_t out_rs,
                            const int32_t *pos, int n_rows, int batch, int n_kv_heads, int head_dim,
                            int32_t *status, void *stream) {
    return q4_store_impl(dt, const_cast<void *>(cache), cache_rs, cache_head_stride, cache_seq_stride, capacity,
                         nullptr, nullptr, k_out, v_out, out_rs, pos, n_rows, batch, n_kv_heads, head_dim, true,
                         status, stream);
}

size_t lat_attn_decode_q4_workspace_size(lat_dtype dt, int batch, int n_heads, int n_kv_heads, int head_dim,
                                         int max_kv_len) {
    if ((dt != LAT_F32 && dt != LAT_BF16) || batch < 0 || batch > 65535 || n_heads <= 0 || n_kv_heads <= 0 ||
        n_heads % n_kv_heads != 0 || !supported_head_dim(head_dim) || !query_row_ok(n_heads, head_dim) ||
        max_kv_len < 0)
        return 0;
    int sms = 0;
    lat::Q4Plan plan;
    if (!current_sm_count(&sms) ||
        !lat::plan_decode_q4(batch, n_heads, n_kv_heads, head_dim, dt == LAT_BF16, max_kv_len, sms, &plan))
        return 0;
    return plan.total_bytes;
}

lat_status lat_attn_decode_q4(lat_dtype dt, const void *q, int64_t q_rs, const void *cache, int64_t cache_rs,
                              int64_t cache_head_stride, int64_t cache_seq_stride, const int32_t *kv_lens,
                              int max_kv_len, void *out, int64_t out_rs, float *lse, int batch, int n_heads,
                              int n_kv_heads, int head_dim, int window, float scale, float softcap,
                              void *workspace, size_t workspace_bytes, int32_t *status, void *stream) {
    return q4_decode_impl(dt, q, q_rs, cache, cache_rs, cache_head_stride, cache_seq_stride, kv_lens, max_kv_len, out,
                          out_rs, lse, batch, n_heads, n_kv_heads, head_dim, window, scale, softcap, workspace,
                          workspace_bytes, status, stream, kDefaultTimeoutNs, 0);
}

lat_status lat_test_decode_q4_timeout(lat_dtype dt, const void *q, int64_t q_rs, const void *cache, int64_t cache_rs,
                                      int64_t cache_head_stride, int64_t cache_seq_stride, const int32_t *kv_lens,
                                      int max_kv_len, void *out, int64_t out_rs, int batch, int n_heads,
                                      int n_kv_heads, int head_dim, void *workspace, size_t workspace_bytes,
                                      uint64_t timeout_ns, int32_t *status, void *stream) {
    return q4_decode_impl(dt, q, q_rs, cache, cache_rs, cache_head_stride, cache_seq_stride, kv_lens, max_kv_len, out,
                          out_rs, nullptr, batch, n_heads, n_kv_heads, head_dim, 0, 0.125f, 0.f, workspace,
                          workspace_bytes, status, stream, timeout_ns, 1);
}

}  // extern "C"

// ---------------------------------------------------------------- the 8-bit cache

namespace {

lat_status q8_store_impl(lat_dtype dt, void *cache, int64_t cache_block_stride, int64_t cache_head_stride,
                         int64_t cache_seq_stride, int block_size, int capacity, const void *k, const void *v,
                         void *k_out, void *v_out, int64_t rs, const int32_t *pos, int n, int batch, int n_kv_heads,
                         int head_dim, bool expand, int32_t *status, void *stream) {
    if (dt != LAT_F32 && dt != LAT_BF16) return LAT_ERR_INVALID_ARG;
    if (batch < 0 || n < 0 || capacity < 0 || n_kv_heads <= 0 || !lat::q8_block_size_ok(block_size))
        return LAT_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim)) return LAT_ERR_UNSUPPORTED;
    if (batch == 0 || n == 0) return LAT_OK;
    if (!cache || !pos || (expand ? (!k_out || !v_out) : (!k || !v))) return LAT_ERR_INVALID_ARG;
    if (!aligned16(cache) || !q4_strides_ok(cache_block_stride, cache_head_stride, cache_seq_stride) ||
        rs < (int64_t)n_kv_heads * head_dim)
        return LAT_ERR_INVALID_ARG;
    const int64_t touched = ((int64_t)n + block_size - 2) / block_size + 1;
    const int64_t per = expand ? n : 2 * touched;  // units of a sequence's head
    if (per * batch > 0x7fffffffLL / n_kv_heads) return LAT_ERR_UNSUPPORTED;
    lat::Q8StoreArgs a{};
    a.cache = static_cast<unsigned char *>(cache);
    a.cache_block = cache_block_stride;
    a.cache_head = cache_head_stride;
    a.cache_seq = cache_seq_stride;
    while (1 << a.block_shift < block_size) ++a.block_shift;
    a.k = k;
    a.v = v;
    a.k_out = k_out;
    a.v_out = v_out;
    a.rs = rs;
    const int64_t es = dt == LAT_BF16 ? 2 : 4;
    a.vec = rs * es % 16 == 0 && (expand ? aligned16(k_out) && aligned16(v_out) : aligned16(k) && aligned16(v));
    a.pos = pos;
    a.capacity = capacity;
    a.n = n;
    a.batch = batch;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.touched = (int)touched;
    a.units = per * batch * n_kv_heads;
    a.by_heads = lat::FastDiv((uint32_t)n_kv_heads);
    a.by_n = lat::FastDiv((uint32_t)n);
    a.by_touched = lat::FastDiv((uint32_t)touched);
    a.status = status;
    return lat::launch_q8_store(a, dt == LAT_BF16, expand, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? LAT_OK
               : LAT_ERR_CUDA;
}

lat_status q8_decode_impl(lat_dtype dt, const void *q, int64_t q_rs, const void *cache, int64_t cache_block_stride,
                          int64_t cache_head_stride, int64_t cache_seq_stride, int block_size,
                          const int32_t *kv_lens, int max_kv_len, void *out, int64_t out_rs, float *lse, int batch,
                          int n_heads, int n_kv_heads, int head_dim, int window, float scale, float softcap,
                          void *workspace, size_t workspace_bytes, int32_t *status, void *stream,
                          uint64_t timeout_ns, int skip_load) {
    if (dt != LAT_F32 && dt != LAT_BF16) return LAT_ERR_INVALID_ARG;
    if (!(softcap >= 0.f) || !isfinite(softcap) || !isfinite(scale)) return LAT_ERR_INVALID_ARG;
    if (batch < 0 || max_kv_len < 0 || n_heads <= 0 || n_kv_heads <= 0 || n_heads % n_kv_heads != 0 ||
        !lat::q8_block_size_ok(block_size))
        return LAT_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim)) return LAT_ERR_UNSUPPORTED;
    if (batch == 0) return LAT_OK;
    if (!q || !cache || !kv_lens || !out) return LAT_ERR_INVALID_ARG;
    const int64_t per16 = dt == LAT_BF16 ? 8 : 4;  // elements in 16 bytes
    if (q_rs < (int64_t)n_heads * head_dim || out_rs < (int64_t)n_heads * head_dim || q_rs % per16 ||
        out_rs % per16 || !aligned16(q) || !aligned16(cache) || !aligned16(out) ||
        !q4_strides_ok(cache_block_stride, cache_head_stride, cache_seq_stride))
        return LAT_ERR_INVALID_ARG;
    if (batch > 65535 || !query_row_ok(n_heads, head_dim)) return LAT_ERR_UNSUPPORTED;
    int sms = 0;
    if (!current_sm_count(&sms)) return LAT_ERR_CUDA;
    lat::SplitPlan plan;
    if (!lat::plan_decode_q8(batch, n_heads, n_kv_heads, head_dim, dt == LAT_BF16, max_kv_len, sms, &plan))
        return LAT_ERR_UNSUPPORTED;
    if (workspace == nullptr || workspace_bytes < plan.total_bytes ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return LAT_ERR_WORKSPACE;
    lat::Q8DecodeArgs a{};
    fill_split_args(a, plan, q, q_rs, kv_lens, max_kv_len, out, out_rs, lse, batch, n_heads, n_kv_heads, head_dim,
                    window, scale, softcap, workspace, status, timeout_ns, skip_load);
    a.cache = static_cast<const unsigned char *>(cache);
    a.cache_block = cache_block_stride;
    a.cache_head = cache_head_stride;
    a.cache_seq = cache_seq_stride;
    while (1 << a.block_shift < block_size) ++a.block_shift;
    return lat::launch_decode_q8(a, dt == LAT_BF16, plan, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? LAT_OK
               : LAT_ERR_CUDA;
}

}  // namespace

extern "C" {

int64_t lat_kv_q8_block_bytes(int head_dim, int block_size) {
    return supported_head_dim(head_dim) && lat::q8_block_size_ok(block_size) ? lat::q8_block_bytes(head_dim, block_size) : 0;
}

lat_status lat_kv_append_q8(lat_dtype dt, void *cache, int64_t cache_block_stride, int64_t cache_head_stride,
                            int64_t cache_seq_stride, int block_size, int capacity, const void *k_new,
                            const void *v_new, int64_t new_rs, const int32_t *pos, int n_new, int batch,
                            int n_kv_heads, int head_dim, int32_t *status, void *stream) {
    return q8_store_impl(dt, cache, cache_block_stride, cache_head_stride, cache_seq_stride, block_size, capacity,
                         k_new, v_new, nullptr, nullptr, new_rs, pos, n_new, batch, n_kv_heads, head_dim, false,
                         status, stream);
}

lat_status lat_kv_expand_q8(lat_dtype dt, const void *cache, int64_t cache_block_stride, int64_t cache_head_stride,
                            int64_t cache_seq_stride, int block_size, int capacity, void *k_out, void *v_out,
                            int64_t out_rs, const int32_t *pos, int n_rows, int batch, int n_kv_heads, int head_dim,
                            int32_t *status, void *stream) {
    return q8_store_impl(dt, const_cast<void *>(cache), cache_block_stride, cache_head_stride, cache_seq_stride,
                         block_size, capacity, nullptr, nullptr, k_out, v_out, out_rs, pos, n_rows, batch, n_kv_heads,
                         head_dim, true, status, stream);
}

size_t lat_attn_decode_q8_workspace_size(lat_dtype dt, int batch, int n_heads, int n_kv_heads, int head_dim,
                                         int max_kv_len) {
    if ((dt != LAT_F32 && dt != LAT_BF16) || batch < 0 || batch > 65535 || n_heads <= 0 || n_kv_heads <= 0 ||
        n_heads % n_kv_heads != 0 || !supported_head_dim(head_dim) || !query_row_ok(n_heads, head_dim) ||
        max_kv_len < 0)
        return 0;
    int sms = 0;
    lat::SplitPlan plan;
    if (!current_sm_count(&sms) ||
        !lat::plan_decode_q8(batch, n_heads, n_kv_heads, head_dim, dt == LAT_BF16, max_kv_len, sms, &plan))
        return 0;
    return plan.total_bytes;
}

lat_status lat_attn_decode_q8(lat_dtype dt, const void *q, int64_t q_rs, const void *cache,
                              int64_t cache_block_stride, int64_t cache_head_stride, int64_t cache_seq_stride,
                              int block_size, const int32_t *kv_lens, int max_kv_len, void *out, int64_t out_rs,
                              float *lse, int batch, int n_heads, int n_kv_heads, int head_dim, int window,
                              float scale, float softcap, void *workspace, size_t workspace_bytes, int32_t *status,
                              void *stream) {
    return q8_decode_impl(dt, q, q_rs, cache, cache_block_stride, cache_head_stride, cache_seq_stride, block_size,
                          kv_lens, max_kv_len, out, out_rs, lse, batch, n_heads, n_kv_heads, head_dim, window, scale,
                          softcap, workspace, workspace_bytes, status, stream, kDefaultTimeoutNs, 0);
}

lat_status lat_test_decode_q8_timeout(lat_dtype dt, const void *q, int64_t q_rs, const void *cache,
                                      int64_t cache_block_stride, int64_t cache_head_stride, int64_t cache_seq_stride,
                                      int block_size, const int32_t *kv_lens, int max_kv_len, void *out,
                                      int64_t out_rs, int batch, int n_heads, int n_kv_heads, int head_dim,
                                      void *workspace, size_t workspace_bytes, uint64_t timeout_ns, int32_t *status,
                                      void *stream) {
    return q8_decode_impl(dt, q, q_rs, cache, cache_block_stride, cache_head_stride, cache_seq_stride, block_size,
                          kv_lens, max_kv_len, out, out_rs, nullptr, batch, n_heads, n_kv_heads, head_dim, 0, 0.125f,
                          0.f, workspace, workspace_bytes, status, stream, timeout_ns, 1);
}

}  // extern "C"

// ---------------------------------------------------------------- weights of cached keys

namespace {

// 4-D bf16 map over query rows: (head-dim d, query head, row, sequence), boxes of box_heads heads of
// box_rows rows, 128-byte swizzle
bool make_columns_map(CUtensorMap *m, const void *base, int head_dim, int heads, int rows, int batch,
                      int64_t row_stride, int box_heads, int box_rows) {
    EncodeTiledFn fn = encode_tiled_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)head_dim, (cuuint64_t)heads, (cuuint64_t)rows, (cuuint64_t)batch};
    const cuuint64_t strides[3] = {(cuuint64_t)head_dim * 2, (cuuint64_t)row_stride * 2,
                                   (cuuint64_t)row_stride * 2 * (cuuint64_t)rows};
    const cuuint32_t box[4] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

lat_status key_weights_impl(lat_dtype dt, const void *q, int64_t q_rs, int n_q, const void *k_cache, int64_t cache_rs,
                            int64_t cache_head_stride, int64_t cache_seq_stride, const int32_t *kv_lens,
                            int max_kv_len, const float *lse, float *weights, int64_t weights_head_stride,
                            int64_t weights_seq_stride, int batch, int n_heads, int n_kv_heads, int head_dim,
                            int causal, int window, float scale, float softcap, int32_t *status, void *stream,
                            uint64_t timeout_ns, int skip_load) {
    if (dt != LAT_F32 && dt != LAT_BF16) return LAT_ERR_INVALID_ARG;
    if (!(softcap >= 0.f) || !isfinite(softcap) || !isfinite(scale)) return LAT_ERR_INVALID_ARG;
    if (batch < 0 || n_q < 0 || max_kv_len < 0 || n_heads <= 0 || n_kv_heads <= 0 || n_heads % n_kv_heads != 0)
        return LAT_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim)) return LAT_ERR_UNSUPPORTED;
    if (batch == 0 || n_q == 0) return LAT_OK;
    if (!q || !k_cache || !kv_lens || !lse || !weights) return LAT_ERR_INVALID_ARG;
    if (q_rs < (int64_t)n_heads * head_dim || cache_rs <= 0 || cache_head_stride <= 0 || cache_seq_stride <= 0 ||
        weights_head_stride < max_kv_len || weights_seq_stride < max_kv_len)
        return LAT_ERR_INVALID_ARG;
    if (dt == LAT_BF16 && (!aligned16(q) || !aligned16(k_cache) || q_rs % 8 || cache_rs % 8 || cache_head_stride % 8 ||
                           cache_seq_stride % 8))
        return LAT_ERR_INVALID_ARG;
    // (the kernels count to the end of a key's tile, and a key behind it, in int)
    if (max_kv_len > 0x7fffff80 || batch > 65535 || !query_row_ok(n_heads, head_dim) ||
        (int64_t)batch * n_q > 0x7fffffffLL || ((int64_t)max_kv_len + 127) / 128 * n_kv_heads > 0x7fffffffLL / batch)
        return LAT_ERR_UNSUPPORTED;
    lat::KeyWeightsArgs a{};
    a.q = q;
    a.k = k_cache;
    a.q_rs = q_rs;
    a.k_row = cache_rs;
    a.k_head = cache_head_stride;
    a.k_seq = cache_seq_stride;
    a.kv_lens = kv_lens;
    a.max_kv_len = max_kv_len;
    a.lse = lse;
    a.weights = weights;
    a.w_seq = weights_seq_stride;
    a.w_head = weights_head_stride;
    a.batch = batch;
    a.n_q = n_q;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.causal = causal != 0;
    a.window = window > 0 && window < max_kv_len ? window : 0;  // (a wider one hides nothing)
    a.scale_log2 = scale * kLog2e;
    softcap = cap_in_range(softcap);
    a.cap_log2 = softcap > 0.f ? softcap * kLog2e : 0.f;
    a.raw_over_cap = softcap > 0.f ? over_cap(scale, softcap) : 0.f;
    a.timeout_ns = timeout_ns;
    a.test_skip_load = skip_load;
    a.status = status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int sms = 0;
    if (dt == LAT_F32) {
        if ((int64_t)batch * n_kv_heads > 65535 || (int64_t)n_q * (n_heads / n_kv_heads) > 0x7fffffffLL)
            return LAT_ERR_UNSUPPORTED;
        a.by_heads_per = lat::FastDiv((uint32_t)(n_heads / n_kv_heads));
        a.q_vec = aligned16(q) && q_rs % 4 == 0;
        a.k_vec = aligned16(k_cache) && cache_rs % 4 == 0 && cache_head_stride % 4 == 0 && cache_seq_stride % 4 == 0;
        if (!current_sm_count(&sms)) return LAT_ERR_CUDA;
        return lat::launch_key_weights_f32(a, sms, s) == cudaSuccess ? LAT_OK : LAT_ERR_CUDA;
    }
    if (!current_sm_count(&sms)) return LAT_ERR_CUDA;
    lat::KeyWeightsPlan plan;
    if (!lat::plan_key_weights(batch, n_q, n_heads, n_kv_heads, head_dim, max_kv_len, sms, &plan))
        return LAT_ERR_UNSUPPORTED;
    a.keys_held = plan.keys_held;
    a.heads_per = plan.heads_per;
    a.by_heads_per = lat::FastDiv((uint32_t)plan.heads_per);
    a.rows_per = plan.rows_per;
    a.head_blocks = plan.head_blocks;
    a.n_cols = plan.n_cols;
    a.slots = plan.slots;
    if (max_kv_len > 0 &&
        (!make_columns_map(&a.tm_q, q, head_dim, n_heads, n_q, batch, q_rs, plan.heads_per, plan.rows_per) ||
         !make_cache_map(&a.tm_k, k_cache, head_dim, n_kv_heads, max_kv_len, batch, cache_rs, cache_head_stride,
                         cache_seq_stride, 128)))
        return LAT_ERR_CUDA;
    return lat::launch_key_weights(a, plan.grid, s) == cudaSuccess ? LAT_OK : LAT_ERR_CUDA;
}

}  // namespace

extern "C" {

lat_status lat_attn_key_weights(lat_dtype dt, const void *q, int64_t q_rs, int n_q, const void *k_cache,
                                int64_t cache_rs, int64_t cache_head_stride, int64_t cache_seq_stride,
                                const int32_t *kv_lens, int max_kv_len, const float *lse, float *weights,
                                int64_t weights_head_stride, int64_t weights_seq_stride, int batch, int n_heads,
                                int n_kv_heads, int head_dim, int causal, int window, float scale, float softcap,
                                int32_t *status, void *stream) {
    return key_weights_impl(dt, q, q_rs, n_q, k_cache, cache_rs, cache_head_stride, cache_seq_stride, kv_lens,
                            max_kv_len, lse, weights, weights_head_stride, weights_seq_stride, batch, n_heads,
                            n_kv_heads, head_dim, causal, window, scale, softcap, status, stream, kDefaultTimeoutNs, 0);
}

lat_status lat_test_key_weights_timeout(const void *q, int64_t q_rs, int n_q, const void *k_cache, int64_t cache_rs,
                                        int64_t cache_head_stride, int64_t cache_seq_stride, const int32_t *kv_lens,
                                        int max_kv_len, const float *lse, float *weights, int64_t weights_head_stride,
                                        int64_t weights_seq_stride, int batch, int n_heads, int n_kv_heads,
                                        int head_dim, uint64_t timeout_ns, int32_t *status, void *stream) {
    return key_weights_impl(LAT_BF16, q, q_rs, n_q, k_cache, cache_rs, cache_head_stride, cache_seq_stride, kv_lens,
                            max_kv_len, lse, weights, weights_head_stride, weights_seq_stride, batch, n_heads,
                            n_kv_heads, head_dim, 1, 0, 0.125f, 0.f, status, stream, timeout_ns, 1);
}

}  // extern "C"

// ---------------------------------------------------------------- eviction

extern "C" {

lat_status lat_kv_evict_choose(const float *weights, int64_t weights_head_stride, int64_t weights_seq_stride,
                               const int32_t *kv_lens, int max_kv_len, int32_t *kept, int n_keep, int n_first,
                               int n_last, float *weights_out, int64_t out_head_stride, int64_t out_seq_stride,
                               int32_t *new_lens, int batch, int n_kv_heads, int32_t *status, void *stream) {
    if (batch < 0 || max_kv_len < 0 || n_kv_heads <= 0 || n_keep < 1 || n_first < 0 || n_last < 0 ||
        (int64_t)n_first + n_last > n_keep)
        return LAT_ERR_INVALID_ARG;
    if (batch == 0) return LAT_OK;
    if (!weights || !kv_lens || !kept || !new_lens || new_lens == kv_lens || weights_head_stride < max_kv_len ||
        weights_seq_stride < max_kv_len)
        return LAT_ERR_INVALID_ARG;
    // one layout where the weights are written over, or rows would meet other rows' entries
    if (weights_out != nullptr &&
        (out_head_stride < max_kv_len || out_seq_stride < max_kv_len ||
         (weights_out == weights && (out_head_stride != weights_head_stride || out_seq_stride != weights_seq_stride))))
        return LAT_ERR_INVALID_ARG;
    if (max_kv_len > lat::kEvictMaxKeys || (int64_t)batch * n_kv_heads > 0x7fffffffLL / lat::kEvictCluster)
        return LAT_ERR_UNSUPPORTED;
    int sms = 0;
    if (!current_sm_count(&sms)) return LAT_ERR_CUDA;
    lat::EvictChooseArgs a{};
    a.weights = weights;
    a.w_seq = weights_seq_stride;
    a.w_head = weights_head_stride;
    a.kv_lens = kv_lens;
    a.max_kv_len = max_kv_len;
    a.kept = kept;
    a.n_keep = n_keep;
    a.n_first = n_first;
    a.n_last = n_last;
    a.out = weights_out;
    a.out_seq = out_seq_stride;
    a.out_head = out_head_stride;
    a.new_lens = new_lens;
    a.batch = batch;
    a.n_kv_heads = n_kv_heads;
    a.status = status;
    return lat::launch_evict_choose(a, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? LAT_OK : LAT_ERR_CUDA;
}

}  // extern "C"

namespace {

lat_status evict_rows_impl(lat_dtype dt, void *k_cache, void *v_cache, int64_t cache_rs, int64_t cache_head_stride,
                           int64_t cache_seq_stride, int capacity, const int32_t *kept, int n_keep, int batch,
                           int n_kv_heads, int head_dim, int32_t *status, void *stream, uint64_t timeout_ns,
                           int skip_tell) {
    if (dt != LAT_F32 && dt != LAT_BF16) return LAT_ERR_INVALID_ARG;
    if (batch < 0 || capacity < 0 || n_keep < 1 || n_kv_heads <= 0) return LAT_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim)) return LAT_ERR_UNSUPPORTED;
    if (batch == 0) return LAT_OK;
    const int es = dt == LAT_BF16 ? 2 : 4;
    auto countable = [](int64_t stride) { return stride > 0 && stride <= INT64_MAX / 4; };  // in bytes, too
    if (!countable(cache_rs) || !countable(cache_head_stride) || !countable(cache_seq_stride) || !k_cache || !v_cache ||
        !kept || !aligned16(k_cache) || !aligned16(v_cache) ||
        !q4_strides_ok(cache_rs * es, cache_head_stride * es, cache_seq_stride * es))
        return LAT_ERR_INVALID_ARG;
    if ((int64_t)batch * n_kv_heads > 0x7fffffffLL / 16) return LAT_ERR_UNSUPPORTED;
    int sms = 0;
    if (!current_sm_count(&sms)) return LAT_ERR_CUDA;
    lat::EvictRowsArgs a{};
    a.k = k_cache;
    a.v = v_cache;
    a.cache_rs = cache_rs * es;
    a.cache_head = cache_head_stride * es;
    a.cache_seq = cache_seq_stride * es;
    a.row_bytes = head_dim * es;
    a.capacity = capacity;
    a.kept = kept;
    a.n_keep = n_keep;
    a.batch = batch;
    a.n_kv_heads = n_kv_heads;
    a.timeout_ns = timeout_ns;
    a.test_skip_tell = skip_tell;
    a.status = status;
    return lat::launch_evict_rows(a, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? LAT_OK : LAT_ERR_CUDA;
}

}  // namespace

extern "C" {

lat_status lat_kv_evict_rows(lat_dtype dt, void *k_cache, void *v_cache, int64_t cache_rs, int64_t cache_head_stride,
                             int64_t cache_seq_stride, int capacity, const int32_t *kept, int n_keep, int batch,
                             int n_kv_heads, int head_dim, int32_t *status, void *stream) {
    return evict_rows_impl(dt, k_cache, v_cache, cache_rs, cache_head_stride, cache_seq_stride, capacity, kept, n_keep,
                           batch, n_kv_heads, head_dim, status, stream, kDefaultTimeoutNs, 0);
}

lat_status lat_test_evict_rows_timeout(lat_dtype dt, void *k_cache, void *v_cache, int64_t cache_rs,
                                       int64_t cache_head_stride, int64_t cache_seq_stride, int capacity,
                                       const int32_t *kept, int n_keep, int batch, int n_kv_heads, int head_dim,
                                       uint64_t timeout_ns, int32_t *status, void *stream) {
    return evict_rows_impl(dt, k_cache, v_cache, cache_rs, cache_head_stride, cache_seq_stride, capacity, kept, n_keep,
                           batch, n_kv_heads, head_dim, status, stream, timeout_ns, 1);
}

}  // extern "C"

// ---------------------------------------------------------------- choice of cached blocks

namespace {

bool block_size_ok(int block_size) { return block_size >= 16 && block_size <= 1024 && block_size % 16 == 0; }

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

// blocks that max_kv_len keys fill
int64_t max_blocks_of(int max_kv_len, int block_size) { return ((int64_t)max_kv_len + block_size - 1) / block_size; }

}  // namespace

extern "C" {

lat_status lat_kv_block_bounds(lat_dtype dt, const void *k_cache, int64_t cache_rs, int64_t cache_head_stride,
                               int64_t cache_seq_stride, int capacity, void *bounds, int64_t bounds_rs,
                               int64_t bounds_head_stride, int64_t bounds_seq_stride, int block_size,
                               const int32_t *pos, int n_new, int batch, int n_kv_heads, int head_dim,
                               int32_t *status, void *stream) {
    if (dt != LAT_F32 && dt != LAT_BF16) return LAT_ERR_INVALID_ARG;
    if (batch < 0 || n_new < 0 || capacity < 0 || n_kv_heads <= 0 || !block_size_ok(block_size))
        return LAT_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim)) return LAT_ERR_UNSUPPORTED;
    if (batch == 0 || n_new == 0) return LAT_OK;
    if (!k_cache || !bounds || !pos) return LAT_ERR_INVALID_ARG;
    const int64_t per16 = dt == LAT_BF16 ? 8 : 4;  // elements in 16 bytes
    if (!aligned16(k_cache) || !aligned16(bounds) || cache_rs <= 0 || cache_head_stride <= 0 ||
        cache_seq_stride <= 0 || bounds_rs <= 0 || bounds_head_stride <= 0 || bounds_seq_stride <= 0 ||
        cache_rs % per16 || cache_head_stride % per16 || cache_seq_stride % per16 || bounds_rs % per16 ||
        bounds_head_stride % per16 || bounds_seq_stride % per16)
        return LAT_ERR_INVALID_ARG;
    // n_new rows touch at most this many blocks, wherever they begin
    const int64_t touched = ((int64_t)n_new + block_size - 2) / block_size + 1;
    if ((int64_t)batch * touched > 0x7fffffffLL / n_kv_heads) return LAT_ERR_UNSUPPORTED;
    lat::BoundsArgs a{};
    a.k_cache = k_cache;
    a.cache_rs = cache_rs;
    a.cache_head = cache_head_stride;
    a.cache_seq = cache_seq_stride;
    a.bounds = bounds;
    a.bounds_rs = bounds_rs;
    a.bounds_head = bounds_head_stride;
    a.bounds_seq = bounds_seq_stride;
    a.block_size = block_size;
    a.capacity = capacity;
    a.n_new = n_new;
    a.max_touched = (int)touched;
    a.batch = batch;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.pos = pos;
    a.status = status;
    return lat::launch_block_bounds(a, dt == LAT_BF16, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? LAT_OK
               : LAT_ERR_CUDA;
}

size_t lat_attn_select_blocks_workspace_size(int batch, int n_kv_heads, int block_size, int max_kv_len) {
    if (batch < 0 || n_kv_heads <= 0 || max_kv_len < 0 || !block_size_ok(block_size) ||
        max_blocks_of(max_kv_len, block_size) > lat::kSelectMaxBlocks)
        return 0;
    const size_t n = (size_t)batch * n_kv_heads * (size_t)max_blocks_of(max_kv_len, block_size);
    return round256(n * sizeof(float2)) + round256(n * sizeof(uint64_t));
}

lat_status lat_attn_select_blocks(lat_dtype dt, const void *q, int64_t q_rs, const void *bounds, int64_t bounds_rs,
                                  int64_t bounds_head_stride, int64_t bounds_seq_stride, int block_size,
                                  const int32_t *kv_lens, int max_kv_len, int32_t *blocks, int n_sel, int n_first,
                                  int n_last, int batch, int n_heads, int n_kv_heads, int head_dim,
                                  void *workspace, size_t workspace_bytes, int32_t *status, void *stream) {
    if (dt != LAT_F32 && dt != LAT_BF16) return LAT_ERR_INVALID_ARG;
    if (batch < 0 || max_kv_len < 0 || n_heads <= 0 || n_kv_heads <= 0 || n_heads % n_kv_heads != 0 ||
        !block_size_ok(block_size) || n_sel <= 0 || n_first < 0 || n_last < 0 || n_first > n_sel ||
        n_last > n_sel - n_first)
        return LAT_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim)) return LAT_ERR_UNSUPPORTED;
    if (batch == 0) return LAT_OK;
    if (!q || !bounds || !kv_lens || !blocks) return LAT_ERR_INVALID_ARG;
    const int64_t per16 = dt == LAT_BF16 ? 8 : 4;
    if (!aligned16(q) || !aligned16(bounds) || q_rs < (int64_t)n_heads * head_dim || q_rs % per16 || bounds_rs <= 0 ||
        bounds_head_stride <= 0 || bounds_seq_stride <= 0 || bounds_rs % per16 || bounds_head_stride % per16 ||
        bounds_seq_stride % per16)
        return LAT_ERR_INVALID_ARG;
    const int64_t max_blocks = max_blocks_of(max_kv_len, block_size);
    if (max_blocks > lat::kSelectMaxBlocks || (int64_t)batch > 0x7fffffffLL / n_kv_heads ||
        !query_row_ok(n_heads, head_dim))
        return LAT_ERR_UNSUPPORTED;
    const size_t need = lat_attn_select_blocks_workspace_size(batch, n_kv_heads, block_size, max_kv_len);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0))
        return LAT_ERR_WORKSPACE;
    int sms = 0;
    if (!current_sm_count(&sms)) return LAT_ERR_CUDA;
    lat::SelectArgs a{};
    a.q = q;
    a.q_rs = q_rs;
    a.bounds = bounds;
    a.bounds_rs = bounds_rs;
    a.bounds_head = bounds_head_stride;
    a.bounds_seq = bounds_seq_stride;
    a.block_size = block_size;
    a.kv_lens = kv_lens;
    a.max_kv_len = max_kv_len;
    a.blocks = blocks;
    a.n_sel = n_sel;
    a.n_first = n_first;
    a.n_last = n_last;
    a.batch = batch;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    const size_t n = (size_t)batch * n_kv_heads * (size_t)max_blocks;
    a.scores = static_cast<float2 *>(workspace);
    a.exact = reinterpret_cast<uint64_t *>(static_cast<unsigned char *>(workspace) + round256(n * sizeof(float2)));
    a.max_blocks = (int)max_blocks;
    a.status = status;
    return lat::launch_select_blocks(a, dt == LAT_BF16, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? LAT_OK
               : LAT_ERR_CUDA;
}

size_t lat_attn_decode_blocks_workspace_size(lat_dtype dt, int batch, int n_heads, int n_kv_heads, int head_dim,
                                             int block_size, int n_sel) {
    if ((dt != LAT_F32 && dt != LAT_BF16) || batch < 0 || batch > 65535 || n_heads <= 0 || n_kv_heads <= 0 ||
        n_heads % n_kv_heads != 0 || !supported_head_dim(head_dim) || !query_row_ok(n_heads, head_dim) ||
        !block_size_ok(block_size) || n_sel <= 0 || n_sel > lat::kSelectMaxBlocks)
        return 0;
    int sms = 0;
    if (!current_sm_count(&sms)) return 0;
    lat::DecodePlan plan;
    if (dt == LAT_BF16)
        return lat::plan_decode_blocks_bf16(batch, n_heads, n_kv_heads, head_dim, n_sel * block_size, sms, &plan)
                   ? plan.total_bytes
                   : 0;
    const size_t rows = (size_t)batch * n_heads;
    const size_t splits = lat::blocks_f32_splits(batch, n_heads, n_kv_heads, block_size, n_sel, sms);
    return splits == 1 ? 256 : round256(rows * splits * head_dim * 4) + round256(rows * splits * 4) + round256(rows * 4);
}

lat_status lat_attn_decode_blocks(lat_dtype dt, const void *q, int64_t q_rs, const void *k_cache,
                                  const void *v_cache, int64_t cache_rs, int64_t cache_head_stride,
                                  int64_t cache_seq_stride, const int32_t *kv_lens, int max_kv_len,
                                  int block_size, const int32_t *blocks, int n_sel, void *out, int64_t out_rs,
                                  float *lse, int batch, int n_heads, int n_kv_heads, int head_dim, float scale,
                                  float softcap, void *workspace, size_t workspace_bytes, int32_t *status,
                                  void *stream) {
    if (dt != LAT_F32 && dt != LAT_BF16) return LAT_ERR_INVALID_ARG;
    if (!block_size_ok(block_size) || n_sel <= 0) return LAT_ERR_INVALID_ARG;
    if (n_sel > lat::kSelectMaxBlocks) return LAT_ERR_UNSUPPORTED;
    if (n_heads > 0 && supported_head_dim(head_dim) && !query_row_ok(n_heads, head_dim)) return LAT_ERR_UNSUPPORTED;
    if (batch > 0 && !blocks) return LAT_ERR_INVALID_ARG;
    if (isfinite(softcap)) softcap = cap_in_range(softcap);  // (others are refused below)
    if (dt == LAT_BF16)
        return decode_impl(dt, q, q_rs, k_cache, v_cache, cache_rs, cache_head_stride, cache_seq_stride, kv_lens,
                           max_kv_len, out, out_rs, lse, batch, n_heads, n_kv_heads, head_dim, 0, scale, softcap, 0,
                           workspace, workspace_bytes, status, stream, kDefaultTimeoutNs, 0, blocks, n_sel,
                           block_size);
    if (!(softcap >= 0.f) || !isfinite(softcap) || !isfinite(scale)) return LAT_ERR_INVALID_ARG;
    if (batch < 0 || max_kv_len < 0 || n_heads <= 0 || n_kv_heads <= 0 || n_heads % n_kv_heads != 0)
        return LAT_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim)) return LAT_ERR_UNSUPPORTED;
    if (batch == 0) return LAT_OK;
    if (!q || !k_cache || !v_cache || !kv_lens || !out) return LAT_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
        q_rs < (int64_t)n_heads * head_dim || out_rs < (int64_t)n_heads * head_dim || q_rs % 4 || out_rs % 4 ||
        cache_rs <= 0 || cache_head_stride <= 0 || cache_seq_stride <= 0 || cache_rs % 4 || cache_head_stride % 4 ||
        cache_seq_stride % 4)
        return LAT_ERR_INVALID_ARG;
    // (a grid has one CTA per sequence, head and up to 128 channels at most, or six per SM)
    if (batch > 65535 || (int64_t)batch * n_heads * ((head_dim + 127) / 128) > 0x7fffffffLL)
        return LAT_ERR_UNSUPPORTED;
    const size_t need = lat_attn_decode_blocks_workspace_size(dt, batch, n_heads, n_kv_heads, head_dim, block_size, n_sel);
    if (need == 0) return LAT_ERR_CUDA;
    if (workspace == nullptr || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return LAT_ERR_WORKSPACE;
    int sms = 0;
    if (!current_sm_count(&sms)) return LAT_ERR_CUDA;
    lat::BlocksF32Args a{};
    a.q = static_cast<const float *>(q);
    a.q_rs = q_rs;
    a.k = static_cast<const float *>(k_cache);
    a.v = static_cast<const float *>(v_cache);
    a.cache_rs = cache_rs;
    a.cache_head = cache_head_stride;
    a.cache_seq = cache_seq_stride;
    a.kv_lens = kv_lens;
    a.max_kv_len = max_kv_len;
    a.blocks = blocks;
    a.n_sel = n_sel;
    a.block_size = block_size;
    a.out = static_cast<float *>(out);
    a.out_rs = out_rs;
    a.lse = lse;
    a.batch = batch;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.head_dim = head_dim;
    a.scale_log2 = scale * kLog2e;
    a.cap_log2 = softcap > 0.f ? softcap * kLog2e : 0.f;
    a.raw_over_cap = softcap > 0.f ? over_cap(scale, softcap) : 0.f;
    a.splits = lat::blocks_f32_splits(batch, n_heads, n_kv_heads, block_size, n_sel, sms);
    const size_t rows = (size_t)batch * n_heads;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    a.part_o = reinterpret_cast<float *>(ws);
    a.part_lse = reinterpret_cast<float *>(ws + round256(rows * a.splits * head_dim * 4));
    a.piece_count = reinterpret_cast<int32_t *>(ws + round256(rows * a.splits * head_dim * 4) + round256(rows * a.splits * 4));
    a.status = status;
    return lat::launch_decode_blocks_f32(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? LAT_OK
                                                                                                   : LAT_ERR_CUDA;
}

lat_status lat_test_decode_blocks_timeout(const void *q, int64_t q_rs, const void *k_cache, const void *v_cache,
                                          int64_t cache_rs, int64_t cache_head_stride, int64_t cache_seq_stride,
                                          const int32_t *kv_lens, int max_kv_len, int block_size,
                                          const int32_t *blocks, int n_sel, void *out, int64_t out_rs, int batch,
                                          int n_heads, int n_kv_heads, int head_dim, void *workspace,
                                          size_t workspace_bytes, uint64_t timeout_ns, int32_t *status,
                                          void *stream) {
    if (!block_size_ok(block_size) || n_sel <= 0 || n_sel > lat::kSelectMaxBlocks || !blocks)
        return LAT_ERR_INVALID_ARG;
    return decode_impl(LAT_BF16, q, q_rs, k_cache, v_cache, cache_rs, cache_head_stride, cache_seq_stride, kv_lens,
                       max_kv_len, out, out_rs, nullptr, batch, n_heads, n_kv_heads, head_dim, 0, 0.125f, 0.f, 0,
                       workspace, workspace_bytes, status, stream, timeout_ns, 1, blocks, n_sel, block_size);
}

}  // extern "C"
