// cache_kernels.h — internal launch interface of the decode operators that read less of a long
// cache: the 4-bit cache and the chosen blocks.  Host-only declarations beside those of
// kernels.h; every argument has been validated by the caller before a launcher runs.
#pragma once

#include <algorithm>
#include <atomic>

#include "kernels.h"

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

// A kernel's dynamic shared memory limit, set once per device (setting it costs a call 1 us).
class SharedLimit {
  public:
    template <typename Kernel>
    cudaError_t operator()(Kernel *k, int smem) {
        int dev = -1;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        std::atomic<bool> *done = dev >= 0 && dev < kDevices ? &done_[dev] : nullptr;
        if (done != nullptr && done->load(std::memory_order_relaxed)) return cudaSuccess;
        e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess && done != nullptr) done->store(true, std::memory_order_relaxed);
        return e;
    }

  private:
    static constexpr int kDevices = 64;
    std::atomic<bool> done_[kDevices] = {};
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

// a split-KV decode over a packed cache (unit_stream.cuh)
struct SplitDecodeArgs {
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
    int max_splits, min_tiles, defer_join, whole;
    uint64_t timeout_ns;
    int test_skip_load;    // test hook: a warp's first copy of a CTA never comes (forces a timeout)
    int32_t *status;
};
struct SplitPlan {
    int grid, whole, min_tiles, max_splits, defer_join;
    size_t part_o_bytes, part_lse_bytes, total_bytes;
};

struct Q4DecodeArgs : SplitDecodeArgs {
    CUtensorMap tm;  // map of 32-bit words over the rows below max_kv_len
};
struct Q4Plan : SplitPlan {
    int wide, twin, box_rows;
};
bool plan_decode_q4(int batch, int n_heads, int n_kv_heads, int head_dim, bool bf16, int max_kv_len, int num_sms,
                    Q4Plan *p);
cudaError_t launch_decode_q4(const Q4DecodeArgs &a, bool bf16, const Q4Plan &p, cudaStream_t s);

// ---------------------------------------------------------------- 8-bit KV cache
struct Q8StoreArgs {
    unsigned char *cache;                        // records (q8_block.cuh); strides in bytes
    int64_t cache_block, cache_head, cache_seq;
    int block_shift;                             // log2 of block_size
    const void *k, *v;                           // append: the new rows
    void *k_out, *v_out;                         // expand: the rows read back
    int64_t rs;                                  // their row stride in elements
    int vec;                                     // 16-byte vectors on that side
    const int32_t *pos;
    int capacity, n, batch, n_kv_heads, head_dim;
    int touched;                                 // append: blocks that n rows can lie in
    int64_t units;                               // append: 2 * batch * touched * n_kv_heads; expand: batch * n * n_kv_heads
    FastDiv by_heads, by_n, by_touched;
    int32_t *status;
};
// units < 2^31
cudaError_t launch_q8_store(const Q8StoreArgs &a, bool bf16, bool expand, cudaStream_t s);

struct Q8DecodeArgs : SplitDecodeArgs {
    const unsigned char *cache;
    int64_t cache_block, cache_head, cache_seq;  // bytes
    int block_shift;
};
bool plan_decode_q8(int batch, int n_heads, int n_kv_heads, int head_dim, bool bf16, int max_kv_len, int num_sms,
                    SplitPlan *p);
cudaError_t launch_decode_q8(const Q8DecodeArgs &a, bool bf16, const SplitPlan &p, cudaStream_t s);

// ---------------------------------------------------------------- weights of cached keys
struct KeyWeightsArgs {
    CUtensorMap tm_q, tm_k;  // bf16: (channel, head, row, sequence), boxes of the plan's columns and of 128 keys
    const void *q, *k;       // fp32
    int64_t q_rs, k_row, k_head, k_seq;  // elements
    int q_vec, k_vec;        // fp32: rows of 16-byte vectors
    const int32_t *kv_lens;
    int max_kv_len;
    const float *lse;        // [batch * n_q, n_heads]
    float *weights;          // key j of (b, hk) at b * w_seq + hk * w_head + j
    int64_t w_seq, w_head;
    int batch, n_q, n_heads, n_kv_heads, head_dim, causal, window;  // window 0: none, else < max_kv_len
    float scale_log2, cap_log2, raw_over_cap;  // as in DecodeArgs
    int keys_held, heads_per, rows_per, head_blocks, n_cols;  // the plan's
    FastDiv by_heads_per;    // fp32: by the KV head's query heads
    int64_t slots;
    uint64_t timeout_ns;
    int test_skip_load;      // test hook: the first stage never comes
    int32_t *status;
};
// A tile of columns is rows_per query rows of heads_per heads (of head_blocks blocks a KV head),
// n_cols of them rounded up to 16.  All columns in one tile: queries held, else keys.
struct KeyWeightsPlan {
    int keys_held, heads_per, rows_per, head_blocks, n_cols, grid;
    int64_t slots;           // key tiles of all sequences, were they as long as they may be
};
bool plan_key_weights(int batch, int n_q, int n_heads, int n_kv_heads, int head_dim, int max_kv_len, int num_sms,
                      KeyWeightsPlan *p);
cudaError_t launch_key_weights(const KeyWeightsArgs &a, int grid, cudaStream_t s);
// batch * n_kv_heads <= 65535
cudaError_t launch_key_weights_f32(const KeyWeightsArgs &a, int num_sms, cudaStream_t s);

// ---------------------------------------------------------------- eviction
constexpr int kEvictCluster = 8, kEvictMaxSlice = 53248;  // CTAs of a head, keys of one in shared memory
constexpr int64_t kEvictMaxKeys = (int64_t)kEvictCluster * kEvictMaxSlice;
struct EvictChooseArgs {
    const float *weights;    // key j of (b, hk) at b * w_seq + hk * w_head + j
    int64_t w_seq, w_head;
    const int32_t *kv_lens;
    int max_kv_len;          // <= kEvictMaxKeys
    int32_t *kept;           // [batch, n_kv_heads, n_keep]
    int n_keep, n_first, n_last;
    float *out;              // nullable; may be weights
    int64_t out_seq, out_head;
    int32_t *new_lens;
    int batch, n_kv_heads, cluster;  // cluster: the launcher's
    int32_t *status;
};
// batch * n_kv_heads * kEvictCluster < 2^31
cudaError_t launch_evict_choose(EvictChooseArgs a, int num_sms, cudaStream_t s);

struct EvictRowsArgs {
    void *k, *v;
    int64_t cache_rs, cache_head, cache_seq;  // bytes
    int row_bytes, capacity;
    const int32_t *kept;                      // [batch, n_kv_heads, n_keep]
    int n_keep, batch, n_kv_heads;
    uint64_t timeout_ns;
    int test_skip_tell;                       // test hook: the first CTA of a cluster does not say that its first rows are there
    int32_t *status;
};
// batch * n_kv_heads * 16 < 2^31
cudaError_t launch_evict_rows(const EvictRowsArgs &a, int num_sms, cudaStream_t s);

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

// ---------------------------------------------------------------- bf16 decode over blocks
// The split-KV decode over the listed blocks alone (window 0, no ring).
struct DecodeBlocksArgs : DecodeArgs {
    const int32_t *blocks;  // [batch, n_kv_heads, n_sel], ascending, -1 behind
    int n_sel, block_size;
};
// Over chosen blocks a CTA's share may be one tile, elsewhere four: with few keys in all, more
// CTAs at once are worth more partials (one sequence, 8 KV heads, 64 blocks of 64 keys: 4 tiles
// 13.6 us, 1 tile 11.2 us; eight sequences: the same).
bool plan_decode_blocks_bf16(int batch, int n_heads, int n_kv_heads, int head_dim, int max_keys, int num_sms,
                             DecodePlan *plan);
cudaError_t launch_decode_blocks_bf16(const DecodeBlocksArgs &a, int grid, cudaStream_t s);

}  // namespace lat
