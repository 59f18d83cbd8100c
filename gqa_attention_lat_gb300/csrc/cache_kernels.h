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
    int max_splits, min_tiles, defer_join, whole;
    uint64_t timeout_ns;
    int test_skip_load;    // test hook: a warp's first copy of a CTA never comes (forces a timeout)
    int32_t *status;
};
struct Q4Plan {
    int grid, wide, twin, whole, min_tiles, max_splits, box_rows, defer_join;
    size_t part_o_bytes, part_lse_bytes, total_bytes;
};
bool plan_decode_q4(int batch, int n_heads, int n_kv_heads, int head_dim, bool bf16, int max_kv_len, int num_sms,
                    Q4Plan *p);
cudaError_t launch_decode_q4(const Q4DecodeArgs &a, bool bf16, const Q4Plan &p, cudaStream_t s);

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
