// kernels.h — internal launch interface between the C-ABI layer (api.cu) and the kernel
// translation units.  Host-only declarations; every argument has been validated by the
// caller before a launcher runs.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

namespace lat {

// Resident CTAs per SM of a kernel as the runtime sees them (shared memory and registers), at
// least 1.  It depends on the kernel and the device alone, so it is asked for once per device:
// the question costs a call 1.4 us.  Sets the kernel's dynamic shared memory limit too.
class Occupancy {
  public:
    template <typename Kernel>
    int operator()(Kernel *k, int threads, int smem) {
        int dev = -1, n = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return 1;
        std::atomic<int> *seen = dev >= 0 && dev < kDevices ? &seen_[dev] : nullptr;
        if (seen != nullptr && (n = seen->load(std::memory_order_relaxed)) > 0) return n;
        if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k, threads, smem) != cudaSuccess)
            return 1;
        n = std::max(1, n);
        if (seen != nullptr) seen->store(n, std::memory_order_relaxed);
        return n;
    }

  private:
    static constexpr int kDevices = 64;
    std::atomic<int> seen_[kDevices] = {};
};

// Division of whole numbers below 2^31 by one fixed beforehand: n / d = (n + hi(n m)) >> s
// (Granlund and Montgomery's round-up multiplier), a handful of instructions where the
// hardware has no divide.
struct FastDiv {
    uint32_t m = 0, s = 0;
    FastDiv() = default;
    explicit FastDiv(uint32_t d) {
        while (s < 31 && (1u << s) < d) ++s;
        m = (uint32_t)(((uint64_t(1) << 32) * ((uint64_t(1) << s) - d)) / d + 1);
    }
#ifdef __CUDACC__
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return (n + __umulhi(n, m)) >> s; }
#endif
};

// ---------------------------------------------------------------- KV-cache append
struct AppendArgs {
    char *k_cache, *v_cache;          // byte pointers
    const char *k_new, *v_new;
    int64_t cache_rs, cache_head, cache_seq, new_rs;  // element strides
    const int32_t *pos;
    int capacity, n_new, batch, n_kv_heads, head_dim, elem_bytes;
    int ring;                         // > 0: position p lives in slot p % ring (no bounds)
    int32_t *status;
};
cudaError_t launch_kv_append(const AppendArgs &a, cudaStream_t s);

// ---------------------------------------------------------------- attention-input producer
// Q/K RMS norm + neox RoPE + V (copy or unit norm) + cache append, one CTA per new row.
struct ProducerArgs {
    const void *qkv;                 // [batch * n_new rows, qkv_rs]: Q heads, K heads, V heads
    int64_t qkv_rs;
    const void *q_w, *k_w;           // [head_dim] norm weights (nullable: weight 1)
    float eps;
    int v_unit_norm;
    void *q_out;                     // [batch * n_new rows, q_out_rs]
    int64_t q_out_rs;
    void *k_cache, *v_cache;
    int64_t cache_rs, cache_head, cache_seq;
    int capacity;
    const int32_t *pos;
    int n_new, batch, n_heads, n_kv_heads, head_dim;
    int32_t *status;
    double inv_freq[256];            // base^(-2i/D), i < head_dim/2, from the host in double
};
cudaError_t launch_qkv_producer(const ProducerArgs &a, bool bf16, cudaStream_t s);

// ---------------------------------------------------------------- fp32 row kernel
// One warp per (query row, query head); used for every fp32 prefill and decode.
// Element (b, j, hk, d) of K is k[b*k_seq + j*k_row + hk*k_head + d] (V alike);
// in decode mode (kv_lens != nullptr) seq_len is 1 and sequence b has kv_lens[b] keys.
struct RowAttnArgs {
    const float *q;
    int64_t q_rs;
    const float *k, *v;
    int64_t k_seq, k_row, k_head, v_seq, v_row, v_head;
    float *out;
    int64_t out_rs;
    float *lse;
    int batch, seq_len, kv_len, n_heads, n_kv_heads, head_dim, causal, window;
    float scale;
    float softcap;                 // > 0: score s becomes softcap * tanh(s / softcap)
    const int32_t *kv_lens;
    int max_kv_len;
    int ring;                      // > 0: key j sits in row j % ring of its sequence
    int32_t *status;
};
cudaError_t launch_row_attention_f32(const RowAttnArgs &a, cudaStream_t s);

// ---------------------------------------------------------------- bf16 split-KV decode
struct DecodeArgs {
    CUtensorMap tm_k, tm_v;  // 4-D maps (d, head, row < max_kv_len, sequence), 128-byte swizzle
    CUtensorMap tm_k16, tm_v16;  // the same with 16-row boxes: a sequence's partial last tile
    CUtensorMap tm_q;        // 3-D map (d, query head, sequence), 8-head boxes, 128-byte swizzle
    const __nv_bfloat16 *q;
    int64_t q_rs;
    const __nv_bfloat16 *k_cache, *v_cache;
    int64_t cache_rs, cache_head, cache_seq;
    const int32_t *kv_lens;
    int max_kv_len;
    __nv_bfloat16 *out;
    int64_t out_rs;
    float *lse;
    int batch, n_heads, n_kv_heads, head_dim, window;
    int ring;           // > 0: ring cache of `ring` rows, key j in row j % ring (window <= ring)
    const int32_t *blocks;  // non-null: only the listed blocks of block_size rows,
    int n_sel, block_size;  // [batch, n_kv_heads, n_sel], ascending, -1 behind
    float scale_log2;   // scale * log2(e): scores are exponentiated with exp2
    float cap_log2, raw_over_cap;  // score cap, as in PrefillTcArgs (cap_log2 0: none)
    // split-KV scratch: partial outputs, partial lse and arrival counters
    float *part_o;      // [batch, n_heads, max_splits, head_dim]
    float *part_lse;    // [batch, n_heads, max_splits]
    int32_t *counters;  // [batch, n_kv_heads, head_blocks]
    int max_splits;  // partial slots per (sequence, KV head, head block)
    int min_seg;     // shortest stretch of one unit's keys a CTA takes (multiple of the tile)
    // few long units: the key stream is cut across every CTA and the pieces are merged by
    // a second kernel; piece_count[b, h] (in the counters' place) tells it how many
    int defer_merge;
    int32_t *piece_count;  // [batch, n_heads] when defer_merge
    int chunked;           // tm_k/tm_v are chunked 5-D maps: one copy per K or V tile
    uint64_t timeout_ns;   // budget of every bounded wait, per CTA
    int test_skip_load;    // test hook: never load a CTA's first K/V stage (forces a timeout)
    int32_t *status;
};
struct DecodePlan {
    int head_blocks, max_splits, min_seg, grid, defer_merge;
    size_t part_o_bytes, part_lse_bytes, counter_bytes, total_bytes;
};
// Chooses the split size and the scratch layout; false when the shape is not built.
bool plan_decode_bf16(int batch, int n_heads, int n_kv_heads, int head_dim, int max_kv_len,
                      int window, int num_sms, DecodePlan *plan, int least_tiles = 4);
// Over chosen blocks a CTA's share may be one tile: with few keys in all, more CTAs at once are
// worth more partials (one sequence, 8 KV heads, 64 blocks of 64 keys: 4 tiles 13.6 us, 1 tile
// 11.2 us; eight sequences: the same).
constexpr int kBlocksLeastTiles = 1;
// work units of one decode launch (sequence x KV head x block of <= 8 query heads); the
// split-KV merge tickets carry a unit index in 23 bits, so plans stop below kDecodeMaxUnits
int64_t decode_bf16_units(int batch, int n_heads, int n_kv_heads);
constexpr int64_t kDecodeMaxUnits = int64_t(1) << 23;
int decode_bf16_tile_keys(int head_dim);     // cache rows per TMA box for this head_dim
cudaError_t launch_decode_bf16(const DecodeArgs &a, int grid, cudaStream_t s);

// ---------------------------------------------------------------- 4-bit KV cache
// bytes of one cached row (a token's K and V of one head), 0 for head sizes not built
int q4_row_bytes(int head_dim);
struct Q4StoreArgs {
    unsigned char *cache;                     // strides in bytes
    int64_t cache_rs, cache_head, cache_seq;
    const void *k, *v;                        // append: the new rows
    void *k_out, *v_out;                      // expand: the rows read back
    int64_t rs;                               // their row stride in elements
    int vec;                                  // 16-byte vectors on that side
    const int32_t *pos;
    int capacity, n, batch, n_kv_heads, head_dim;
    FastDiv by_heads, by_n;                   // by n_kv_heads, by n
    int32_t *status;
};
// batch * n * n_kv_heads < 2^31
cudaError_t launch_q4_store(const Q4StoreArgs &a, bool bf16, bool expand, cudaStream_t s);

struct Q4DecodeArgs {
    CUtensorMap tm;  // map of 32-bit words over the rows below max_kv_len
    const void *q;
    int64_t q_rs;
    const int32_t *kv_lens;
    int max_kv_len;
    void *out;
    int64_t out_rs;
    float *lse;
    int batch, n_heads, n_kv_heads, head_dim, window;
    float scale_log2, cap_log2;  // as in DecodeArgs
    float over_cap_log2;         // 1 / (softcap * log2(e)): a log2-domain score over the cap
    float *part_o;         // [batch, n_heads, max_splits, head_dim]
    float *part_lse;       // [batch, n_heads, max_splits], log2 domain
    int32_t *piece_count;  // defer_join: [batch, n_heads]
    int32_t *counters;     // else: tickets [batch, n_kv_heads, blocks of heads], zero between calls
    int max_splits, min_tiles, defer_join;
    uint64_t timeout_ns;
    int32_t *status;
};
struct Q4Plan {
    int grid, min_tiles, max_splits, box_rows, defer_join;
    size_t part_o_bytes, part_lse_bytes, total_bytes;
};
bool plan_decode_q4(int batch, int n_heads, int n_kv_heads, int head_dim, bool bf16, int max_kv_len, int num_sms,
                    Q4Plan *p);
cudaError_t launch_decode_q4(const Q4DecodeArgs &a, bool bf16, int grid, cudaStream_t s);

// ---------------------------------------------------------------- choice of cached blocks
struct BoundsArgs {
    const void *k_cache;
    int64_t cache_rs, cache_head, cache_seq;  // elements
    void *bounds;                             // row n: D maxima, D minima of block n
    int64_t bounds_rs, bounds_head, bounds_seq;
    int block_size, capacity, n_new, max_touched, batch, n_kv_heads, head_dim;
    const int32_t *pos;
    int32_t *status;
};
// batch * max_touched * n_kv_heads < 2^31
cudaError_t launch_block_bounds(const BoundsArgs &a, bool bf16, cudaStream_t s);

constexpr int kSelectMaxBlocks = 65536;  // a sequence's blocks, a bit each in shared memory
struct SelectArgs {
    const void *q;
    int64_t q_rs;
    const void *bounds;
    int64_t bounds_rs, bounds_head, bounds_seq;
    int block_size;
    const int32_t *kv_lens;
    int max_kv_len;
    int32_t *blocks;  // [batch, n_kv_heads, n_sel]
    int n_sel, n_first, n_last, batch, n_heads, n_kv_heads, head_dim;
    float2 *scores;   // [batch, n_kv_heads, max_blocks]: the score, a bound of its error
    uint64_t *exact;  // [batch, n_kv_heads, max_blocks]: ordered fp64 scores near the border
    int max_blocks, keys_held;
    int32_t *status;
};
cudaError_t launch_select_blocks(SelectArgs a, bool bf16, int num_sms, cudaStream_t s);

// ---------------------------------------------------------------- fp32 decode over blocks
struct BlocksF32Args {
    const float *q;
    int64_t q_rs;
    const float *k, *v;
    int64_t cache_rs, cache_head, cache_seq;
    const int32_t *kv_lens;
    int max_kv_len;
    const int32_t *blocks;
    int n_sel, block_size;
    float *out;
    int64_t out_rs;
    float *lse;
    int batch, n_heads, n_kv_heads, head_dim;
    float scale_log2, cap_log2, raw_over_cap;
    float *part_o, *part_lse;
    int32_t *piece_count;
    int splits;  // pieces of a unit, all of them written
    int32_t *status;
};
// pieces per (sequence, KV head, block of heads)
int blocks_f32_splits(int batch, int n_heads, int n_kv_heads, int block_size, int n_sel, int num_sms);
cudaError_t launch_decode_blocks_f32(const BlocksF32Args &a, cudaStream_t s);

// ---------------------------------------------------------------- bf16 tensor-core prefill
struct PrefillTcArgs {
    CUtensorMap tm_q, tm_k, tm_v;  // 4-D maps (d, head, row, batch), 128-byte swizzle
    // 3-D map over the output (column, row < seq_len, batch), 32-row boxes of
    // prefill_tc_out_box_cols columns; used where that is nonzero
    CUtensorMap tm_out;
    __nv_bfloat16 *out;
    int64_t out_rs;
    int out_v8;                    // out and out_rs allow 32-byte row stores
    float *lse;
    int batch, seq_len, kv_len, n_heads, n_kv_heads, head_dim, causal, window;
    float scale_log2;              // scale * log2(e)
    // score cap: when cap_log2 > 0 a raw dot product x scores cap_log2 * tanh(x * raw_over_cap)
    // in the log2 domain (softcap * log2(e) and scale / softcap), replacing x * scale_log2
    float cap_log2, raw_over_cap;
    int32_t *status;
    uint64_t timeout_ns;
    int test_skip_kv_load;         // test hook: never load KV tile 0 (forces a timeout)
    int wide;                      // head_dim 64: the 96-key-tile form (prefill_tc_wide)
    int pair;                      // head_dim 512, even GQA group: the CTA-pair form
    int chunked;                   // tm_q/k/v are chunked 5-D maps: one copy per tile
};
// the 96-key-tile form of head_dim 64 for long key ranges (a query tile visiting ~1K keys)
bool prefill_tc_wide(int head_dim, int seq_len, int kv_len, int causal, int window);
int prefill_tc_block_n(int head_dim, bool wide);  // keys per KV tile
// head_dim 512 with an even number of query heads per KV head runs on CTA pairs
bool prefill_tc_pair(int head_dim, int n_heads, int n_kv_heads);
// rows of the K (v = false) or V (v = true) tensor-map box of the chosen form
int prefill_tc_box_rows(int head_dim, bool wide, bool pair, bool v);
// forms that move each tile in one copy through chunked 5-D maps, and the 64-column
// chunks of one V copy
bool prefill_tc_chunked(int head_dim, bool pair);
// columns of one output box where the epilogue stores through tm_out, else 0
int prefill_tc_out_box_cols(int head_dim, bool pair);
int prefill_tc_v_chunks(int head_dim, bool pair);
// work items of one prefill launch (query tile x head x output-column part); the kernel
// numbers them in int32, so the host refuses shapes above kPrefillMaxItems
int64_t prefill_tc_items(int batch, int n_heads, int head_dim, int seq_len);
constexpr int64_t kPrefillMaxItems = int64_t(1) << 30;
cudaError_t launch_prefill_tc(const PrefillTcArgs &a, int num_sms, cudaStream_t s);
// out[i] = the capped score (log2 domain) of raw[i], as the bf16 kernels form it
cudaError_t launch_capped_scores(const float *raw, int64_t n, float raw_over_cap,
                                 float cap_log2, float *out, cudaStream_t s);

}  // namespace lat
