// key_weights.cu — what each cached key was given by the last n_q query rows of its sequence.
//
// What it computes, with the log-sum-exp that each row's attention left: for sequence b of length
// L, KV head hk with its G query heads, key j,
//   weights[b, hk, j] += sum_{i < n_q} sum_{g < G} e^{s_ij - lse_i},  s as in the attention calls,
// over the rows i (at positions L - n_q + i >= 0) that see key j.  With the log-sum-exp at hand
// no row needs another key's score: one product of keys and queries, one exponential a pair, one
// sum over a key's pairs.
//
// bf16 (key_weights_kernel):
//  * S^T = K Q^T on tcgen05: 128 keys are M, so that a thread of the epilogue owns a key (a lane
//    of tensor memory) and sums its row in a register: no value passes between threads.  N is up
//    to 256 columns, a column being one (row, query head), which TMA lays side by side from the
//    query rows as they are.
//  * Few columns (they fit one tile next to the ring, a decode step or an observation window):
//    the tile of queries stays in shared memory while key tiles stream by, each read once.  The
//    CTAs take equal shares of all key tiles, a scan over the lengths says which.
//    More columns (a chunk, a prompt): a key tile stays while its tiles of queries stream by, and
//    items (key tiles) are dealt heaviest first, forwards and backwards in turn.
//    Either way every key has one owner, so sums are in a fixed order and nothing is atomic.
//  * Roles: warps 0-3 and 4-7 are two epilogues that take every other tile of S (two buffers in
//    tensor memory), warp 8 issues the copies, warp 9 the MMAs, warp 10 prepares each column's
//    log-sum-exp and range of keys.  Where a range cuts a tile, pairs are masked one by one.
//  * A thread adds a tile's columns in four sums and those to its total with a compensation, so
//    prompts of many thousand rows lose nothing.
//  * Waits are bounded; on expiry the CTA records LAT_ERR_TIMEOUT, drains and quits.
// What bounds it: HBM (keys once) for few columns; for many the tensor pipe and the exponentials,
// 128 N D 2 flops against 128 N of them.
//
// fp32 (key_weights_f32_kernel): exact fp32 products, 64 keys x 8 or 64 columns a step, a thread 4
// x 1 or 4 x 8 of them.  Bound by its FMAs.
#include <math.h>

#include <algorithm>

#include "cache_kernels.h"
#include "device_common.cuh"
#include "score_cap.cuh"
#include "tc_desc.cuh"

namespace lat {

namespace {

constexpr int kKeysTile = 128;
constexpr int kTcThreads = 352;
constexpr int kEpilogueWarps = 8, kCopyWarp = 8, kMmaWarp = 9, kTableWarp = 10;
constexpr int kMaxCols = 256, kStreamCols = 128;  // columns of a tile: at most, and where they stream
constexpr uint32_t kTmemCols = 512;               // two tiles of S

template <int D>
struct KwCfg {
    static constexpr int kChunks = (D + 63) / 64;           // 64-channel chunks of a row
    static constexpr int kSteps = (D + 15) / 16;            // MMAs of a tile
    static constexpr int kStageChunks = D == 64 ? 1 : 2;    // chunks of a ring stage, 16 KB each
    static constexpr int kStagesPerTile = kChunks / kStageChunks;
    static constexpr int kStageBytes = kStageChunks * 16384;
    static constexpr int kStages = D == 512 ? 2 : D == 64 ? 8 : 4;
    // the operand that stays: up to 256 (head_dim 256, 512: 128) columns, or 128 keys
    static constexpr int kHeldBytes = D == 512 ? 131072 : 65536;
    static constexpr int kHeldCols = kHeldBytes / (kChunks * 128) < kMaxCols ? kHeldBytes / (kChunks * 128) : kMaxCols;
    static constexpr int kTableBytes = 2 * (3 * kMaxCols + 4) * 4;
    static constexpr int kBarBytes = 512;
    static constexpr int kSmem = 1024 + kHeldBytes + kStages * kStageBytes + kTableBytes + kKeysTile * 4 + kBarBytes;
    static_assert(kSmem <= 232448, "shared memory budget");
};

// the columns of a tile: e^{s - lse} = 2^(s' - lse2), and the keys lo < j <= hi that a column sees
struct Table {
    float lse2[kMaxCols];
    int hi[kMaxCols], lo[kMaxCols];
    int min_hi, max_lo, count, pad;  // over the columns there are
};

struct Item {
    int b, hk, t;        // key tile
    int len;
    int64_t col0, col1;  // its tiles of columns
    bool fresh;          // another sequence or head than the item before
};

__device__ __forceinline__ int length_of(const KeyWeightsArgs &a, int b) {
    const int len = a.kv_lens[b];
    return len < 0 || len > a.max_kv_len ? 0 : len;
}
// key tiles that some row of a sequence sees
__device__ __forceinline__ int2 tiles_seen(const KeyWeightsArgs &a, int len) {
    const int first = max(0, len - a.n_q);  // the first row's position
    const int lo = a.window > 0 ? max(0, first - a.window + 1) : 0;
    return make_int2(lo / kKeysTile, (int)(((int64_t)len + kKeysTile - 1) / kKeysTile));
}

// The CTA's items.  Queries held: a share of the sequence of (b, hk, t); keys held: every grid-th
// of (t, b, hk), forwards and backwards in turn.
struct Walker {
    const KeyWeightsArgs &a;
    int64_t pos, end;   // next item, and behind the last; or the round
    int64_t base;       // queries held: where sequence b's items begin
    int b, hk, t, t1, len;

    __device__ Walker(const KeyWeightsArgs &a_, int64_t pos_, int64_t end_, int64_t base_, int b_)
        : a(a_), pos(pos_), end(end_), base(base_), b(b_), hk(-1), t(0), t1(0), len(0) {}

    __device__ bool next(Item &it) {
        return a.keys_held ? next_dealt(it) : next_shared(it);
    }
    __device__ bool next_shared(Item &it) {
        if (pos >= end) return false;
        it.fresh = true;
        if (hk >= 0 && t + 1 < t1) {
            ++t;
            it.fresh = false;
        } else {
            for (;;) {  // another head, or sequence
                len = length_of(a, b);
                const int2 seen = tiles_seen(a, len);
                const int64_t n = seen.y - seen.x;
                if (pos >= base + n * a.n_kv_heads) {
                    base += n * a.n_kv_heads;
                    ++b;
                    continue;
                }
                hk = (int)((pos - base) / n);
                t = seen.x + (int)((pos - base) % n);
                t1 = seen.y;
                break;
            }
        }
        ++pos;
        it.b = b, it.hk = hk, it.t = t, it.len = len, it.col0 = 0, it.col1 = 1;
        return true;
    }
    __device__ bool next_dealt(Item &it) {
        const int64_t per = (int64_t)a.batch * a.n_kv_heads;
        for (;; ++pos) {
            const int64_t x = pos * gridDim.x + ((pos & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
            if (pos * gridDim.x >= end) return false;
            if (x >= end) continue;
            it.t = (int)(x / per);
            const int rem = (int)(x - it.t * per);
            it.b = rem / a.n_kv_heads;
            it.hk = rem - it.b * a.n_kv_heads;
            it.len = length_of(a, it.b);
            const int2 seen = tiles_seen(a, it.len);
            if (it.t < seen.x || it.t >= seen.y) continue;
            // rows that see a key of the tile
            const int64_t off = (int64_t)it.len - a.n_q, first = (int64_t)it.t * kKeysTile;
            const int64_t last = min(first + kKeysTile, (int64_t)it.len) - 1;
            int64_t i0 = max((int64_t)0, -off), i1 = a.n_q - 1;
            if (a.causal) i0 = max(i0, first - off);
            if (a.window > 0) i1 = min(i1, last + a.window - 1 - off);
            if (i0 > i1) continue;
            it.col0 = i0 / a.rows_per * a.head_blocks;
            it.col1 = (i1 / a.rows_per + 1) * a.head_blocks;
            it.fresh = true;
            ++pos;
            return true;
        }
    }
};

// sum over 16 columns of 2^(s' - lse2), the scores as they came out of the MMA
template <bool CAP, bool MASK>
__device__ __forceinline__ void add_columns(float (&sum)[4], const uint32_t (&r)[16], const Table &tab, int n0, int j,
                                            const KeyWeightsArgs &a) {
    float x[16];
    if constexpr (CAP) {
        float most = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            x[k] = __uint_as_float(r[k]) * a.raw_over_cap;
            most = fmaxf(most, fabsf(x[k]));
        }
        // scores well below the cap (tanh's Taylor series, as in capped_score_close) are most
        if (__any_sync(0xffffffffu, !(most < 0.3f))) {
#pragma unroll
            for (int k = 0; k < 16; ++k) x[k] = capped_score_close(x[k], a.cap_log2);
        } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const float z = x[k] * x[k];
                const float t = fmaf(z, fmaf(z, fmaf(z, fmaf(z, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f), 1.f);
                x[k] = a.cap_log2 * x[k] * t;
            }
        }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float4 l = *reinterpret_cast<const float4 *>(tab.lse2 + n0 + 4 * q);
        const float ls[4] = {l.x, l.y, l.z, l.w};
        int hi[4], lo[4];
        if constexpr (MASK) {
            const int4 h = *reinterpret_cast<const int4 *>(tab.hi + n0 + 4 * q);
            const int4 o = *reinterpret_cast<const int4 *>(tab.lo + n0 + 4 * q);
            hi[0] = h.x, hi[1] = h.y, hi[2] = h.z, hi[3] = h.w;
            lo[0] = o.x, lo[1] = o.y, lo[2] = o.z, lo[3] = o.w;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float p = fast_exp2(CAP ? x[4 * q + k] - ls[k] : fmaf(__uint_as_float(r[4 * q + k]), a.scale_log2, -ls[k]));
            sum[k] += !MASK || (j <= hi[k] && j > lo[k]) ? p : 0.f;
        }
    }
}

template <int D, bool CAP>
__global__ void __launch_bounds__(kTcThreads, 1) key_weights_kernel(const __grid_constant__ KeyWeightsArgs a) {
    using C = KwCfg<D>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char *held = smem;                                  // one or two operands that stay
    unsigned char *ring = held + C::kHeldBytes;                  // [kStages]
    Table *tables = reinterpret_cast<Table *>(ring + C::kStages * C::kStageBytes);  // [2]
    float *passed = reinterpret_cast<float *>(tables + 2);       // [128] the second epilogue's totals
    uint64_t *bars = reinterpret_cast<uint64_t *>(passed + kKeysTile);
    uint64_t *ring_full = bars, *ring_empty = bars + 8;          // [kStages]
    uint64_t *held_full = bars + 16, *held_empty = bars + 18;    // [2]
    uint64_t *s_full = bars + 20, *s_empty = bars + 22;          // [2]
    uint64_t *tab_full = bars + 24, *tab_empty = bars + 26;      // [2]
    uint64_t *x_full = bars + 28, *x_empty = bars + 32;          // [4] by quarter of the lanes
    uint64_t *bar_done = bars + 36;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 37);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *scan = reinterpret_cast<int *>(tmem_slot + 2);          // [11] warps
    int64_t *start = reinterpret_cast<int64_t *>(bars + 44);     // share: base, b
    static_assert(sizeof(Table) * 2 == C::kTableBytes && C::kStages <= 8, "shared memory layout");

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.n_heads / a.n_kv_heads;
    const uint64_t deadline = globaltimer_ns() + a.timeout_ns;
    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) mbar_init(&ring_full[i], 1), mbar_init(&ring_empty[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&held_full[i], 1), mbar_init(&held_empty[i], 1);
            mbar_init(&s_full[i], 1), mbar_init(&s_empty[i], 4);
            mbar_init(&tab_full[i], 1), mbar_init(&tab_empty[i], kEpilogueWarps);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&x_full[i], 1), mbar_init(&x_empty[i], 1);
        mbar_init(bar_done, 1);
        *abort_flag = 0;
        fence_mbarrier_init();
        start[0] = 0, start[1] = a.batch;
    }
    if (warp == kMmaWarp) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    // ---- this CTA's share: per-thread sums over a slice of the sequences, then a scan ----------
    // (item counts stay below 2^31)
    const int per_thread = (a.batch + kTcThreads - 1) / kTcThreads;
    const int b_lo = min(a.batch, tid * per_thread), b_hi = min(a.batch, b_lo + per_thread);
    int mine = 0;
    for (int b = b_lo; b < b_hi; ++b) {
        const int n = a.kv_lens[b];
        if (blockIdx.x == 0 && (n < 0 || n > a.max_kv_len)) report_status(a.status, kErrBounds);
        const int2 seen = tiles_seen(a, length_of(a, b));
        mine += (seen.y - seen.x) * a.n_kv_heads;
    }
    int incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
    }
    if (lane == 31) scan[warp] = incl;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    int total = 0, before = incl - mine;
    for (int w = 0; w < kTcThreads / 32; ++w) {
        const int v = scan[w];
        if (w < warp) before += v;
        total += v;
    }
    int64_t r0 = 0, r1 = a.slots;
    if (!a.keys_held) {
        const int each = total / (int)gridDim.x, more = total % (int)gridDim.x, c = blockIdx.x;
        r0 = (int64_t)each * c + min(c, more);
        r1 = r0 + each + (c < more ? 1 : 0);
        if (r0 < r1 && r0 >= before && r0 - before < mine) {
            int64_t base = before;
            int b = b_lo;
            for (; b < b_hi; ++b) {
                const int2 seen = tiles_seen(a, length_of(a, b));
                const int64_t n = (int64_t)(seen.y - seen.x) * a.n_kv_heads;
                if (r0 < base + n) break;
                base += n;
            }
            start[0] = base, start[1] = b;
        }
        __syncthreads();
    }
    Walker walk(a, r0, r1, start[0], (int)start[1]);
    // bytes of a chunk of the tile of queries and of keys; how many operands there is room to hold
    const int q_rows = a.rows_per * a.heads_per;                 // columns that a copy brings
    const int q_chunk = a.keys_held ? 16384 : a.n_cols * 128;    // where its chunks lie apart
    const int held_bytes = C::kChunks * (a.keys_held ? 16384 : q_chunk);
    const int n_held = 2 * held_bytes <= C::kHeldBytes ? 2 : 1;
    auto wait = [&](uint64_t *bar, uint32_t parity) { return mbar_wait_bounded(bar, parity, abort_flag, deadline); };

    if (warp == kCopyWarp) {
        if (lane == 0) {
            if (a.max_kv_len > 0) tma_prefetch_desc(&a.tm_q), tma_prefetch_desc(&a.tm_k);  // (else there are none)
            unsigned g = 0, h = 0;  // ring stages and held operands issued
            bool ok = true;
            // chunks [c0, c1) of a tile of keys or of queries (column tile x)
            auto keys = [&](unsigned char *to, uint64_t *bar, const Item &it, int c0, int c1) {
                for (int c = c0; c < c1; ++c)
                    tma_load_4d(to + (c - c0) * 16384, &a.tm_k, bar, c * 64, it.hk, it.t * kKeysTile, it.b);
            };
            auto queries = [&](unsigned char *to, uint64_t *bar, const Item &it, int64_t x, int c0, int c1) {
                const int rb = (int)(x / a.head_blocks), hb = (int)(x % a.head_blocks);
                for (int c = c0; c < c1; ++c)
                    tma_load_4d(to + (c - c0) * q_chunk, &a.tm_q, bar, c * 64, it.hk * G + hb * a.heads_per,
                                rb * a.rows_per, it.b);
            };
            for (Item it; ok && walk.next(it);) {
                if (it.fresh) {
                    const unsigned x = h % n_held;
                    if (!(ok = wait(&held_empty[x], ((h / n_held) & 1) ^ 1))) break;
                    mbar_arrive_expect_tx(&held_full[x], C::kChunks * (a.keys_held ? 16384 : q_rows * 128));
                    if (a.keys_held) keys(held + x * held_bytes, &held_full[x], it, 0, C::kChunks);
                    else queries(held + x * held_bytes, &held_full[x], it, 0, 0, C::kChunks);
                    ++h;
                }
                for (int64_t x = it.col0; ok && x < it.col1; ++x)
                    for (int p = 0; p < C::kStagesPerTile; ++p, ++g) {
                        const unsigned s = g % C::kStages;
                        if (!(ok = wait(&ring_empty[s], ((g / C::kStages) & 1) ^ 1))) break;
                        if (a.test_skip_load && g == 0) continue;  // test hook: never comes
                        const int c0 = p * C::kStageChunks;
                        mbar_arrive_expect_tx(&ring_full[s], C::kStageChunks * (a.keys_held ? q_rows * 128 : 16384));
                        if (a.keys_held) queries(ring + s * C::kStageBytes, &ring_full[s], it, x, c0, c0 + C::kStageChunks);
                        else keys(ring + s * C::kStageBytes, &ring_full[s], it, c0, c0 + C::kStageChunks);
                    }
            }
            // every copy lands before the CTA leaves: slot s last held the largest fill s + k * slots
            const uint64_t until = globaltimer_ns() + 100000000ull;
            volatile int no_abort = 0;
            for (unsigned s = 0; s < C::kStages && s < g; ++s) {
                const unsigned last = s + (g - 1 - s) / C::kStages * C::kStages;
                if (!(a.test_skip_load && last == 0)) mbar_wait_bounded(&ring_full[s], (last / C::kStages) & 1, &no_abort, until);
            }
            for (unsigned s = 0; s < (unsigned)n_held && s < h; ++s) {
                const unsigned last = s + (h - 1 - s) / n_held * n_held;
                mbar_wait_bounded(&held_full[s], (last / n_held) & 1, &no_abort, until);
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        if (lane == 0) {
            const uint32_t idesc = instr_desc(kKeysTile, a.n_cols, false);
            unsigned g = 0, h = 0, step = 0;  // ring stages, held operands, tiles of S
            bool ok = true;
            for (Item it; ok && walk.next(it);) {
                if (it.fresh) {
                    if (h > 0) tc_commit(&held_empty[(h - 1) % n_held]);
                    if (!(ok = wait(&held_full[h % n_held], (h / n_held) & 1))) break;
                    ++h;
                }
                const uint32_t kept = smem_u32(held + (h - 1) % n_held * held_bytes);
                for (int64_t x = it.col0; ok && x < it.col1; ++x, ++step) {
                    if (!(ok = wait(&s_empty[step & 1], ((step >> 1) & 1) ^ 1))) break;
                    const uint32_t d = tmem + (step & 1) * kMaxCols;
                    for (int p = 0; p < C::kStagesPerTile; ++p, ++g) {
                        const unsigned s = g % C::kStages;
                        if (!(ok = wait(&ring_full[s], (g / C::kStages) & 1))) break;
                        tc_fence_after();
                        const uint32_t here = smem_u32(ring + s * C::kStageBytes);
                        // a chunk of keys is 16 KB wherever it lies
                        const uint64_t dk = sw128_desc(a.keys_held ? kept + p * C::kStageChunks * 16384 : here);
                        const uint64_t dq = sw128_desc(a.keys_held ? here : kept + p * C::kStageChunks * q_chunk);
#pragma unroll
                        for (int c = 0; c < C::kStageChunks; ++c)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (D % 64 == 0 || c * 4 + k < C::kSteps)
                                    tc_mma_ss(d, dk + (uint64_t)((c * 16384 + k * 32) >> 4),
                                              dq + (uint64_t)((c * q_chunk + k * 32) >> 4), idesc, p > 0 || c > 0 || k > 0);
                        tc_commit(&ring_empty[s]);
                    }
                    if (ok) tc_commit(&s_full[step & 1]);
                }
            }
            // all MMAs finish before tensor memory is freed
            tc_commit(bar_done);
            volatile int no_abort = 0;
            mbar_wait_bounded(bar_done, 0, &no_abort, globaltimer_ns() + 100000000ull);
        }
        __syncwarp();
    } else if (warp == kTableWarp) {
        unsigned n = 0;  // tables made
        for (Item it; walk.next(it);) {
            if (!a.keys_held && !it.fresh) continue;
            bool ok = true;
            for (int64_t x = it.col0; x < it.col1; ++x, ++n) {
                ok = __all_sync(0xffffffffu, wait(&tab_empty[n & 1], ((n >> 1) & 1) ^ 1));
                if (!ok) break;
                Table &tab = tables[n & 1];
                const int rb = (int)(x / a.head_blocks), hb = (int)(x % a.head_blocks);
                const int rows = min(a.rows_per, a.n_q - rb * a.rows_per), heads = min(a.heads_per, G - hb * a.heads_per);
                // (one block of heads, or one row a tile: the columns there are come first)
                const int count = a.head_blocks == 1 ? rows * heads : heads;
                int min_hi = 0x7fffffff, max_lo = -1;
                for (int i = lane; i < a.n_cols; i += 32) {
                    int hi = -1, lo = -1;
                    float l = INFINITY;
                    if (i < count) {
                        const int row = rb * a.rows_per + i / a.heads_per, pos = it.len - a.n_q + row;
                        l = a.lse[((int64_t)it.b * a.n_q + row) * a.n_heads + it.hk * G + hb * a.heads_per + i % a.heads_per];
                        if (pos >= 0 && l != -INFINITY) {  // (else the row sees nothing)
                            hi = a.causal ? pos : 0x7fffffff;
                            lo = a.window > 0 ? pos - a.window : -1;
                        }
                        l = l == -INFINITY ? INFINITY : l * 1.4426950408889634f;
                        min_hi = min(min_hi, hi);
                        max_lo = max(max_lo, lo);
                    }
                    tab.lse2[i] = l, tab.hi[i] = hi, tab.lo[i] = lo;
                }
                min_hi = __reduce_min_sync(0xffffffffu, min_hi);
                max_lo = __reduce_max_sync(0xffffffffu, max_lo);
                if (lane == 0) tab.min_hi = min_hi, tab.max_lo = max_lo, tab.count = count;
                __syncwarp();
                if (lane == 0) mbar_arrive(&tab_full[n & 1]);
            }
            if (!ok) break;
        }
    } else {
        // ---- epilogues: thread = key ----------------------------------------------------------
        const unsigned group = warp >> 2, quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        auto wait_warp = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
        unsigned step = 0, tabs = 0, items = 0;  // tiles of S, tables, items before this one
        bool ok = true;
        for (Item it; ok && walk.next(it); ++items) {
            const int first = it.t * kKeysTile, j = first + row, last = min(first + kKeysTile, it.len) - 1;
            // keys held: the first epilogue has the last word on every item
            const bool writes = a.keys_held ? group == 0 : (step & 1) == group;
            float *dst = a.weights + (int64_t)it.b * a.w_seq + (int64_t)it.hk * a.w_head + j;
            const float was = writes && j < it.len ? *dst : 0.f;
            float sum = 0.f, lost = 0.f;
            for (int64_t x = it.col0; x < it.col1; ++x, ++step) {
                if (a.keys_held || it.fresh) {  // another table: every warp lets the last go, and has seen
                    if (tabs > 0) {             // each one full before it lets that go
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&tab_empty[(tabs - 1) & 1]);
                    }
                    if (!(ok = wait_warp(&tab_full[tabs & 1], (tabs >> 1) & 1))) break;
                    ++tabs;
                }
                if ((step & 1) != group) continue;
                if (!(ok = wait_warp(&s_full[group], (step >> 1) & 1))) break;
                tc_fence_after();
                const Table &tab = tables[(tabs - 1) & 1];
                const int count = tab.count, whole = count / 16 * 16;
                const bool mask = tab.min_hi < last || tab.max_lo >= first;
                const uint32_t src = lanes + group * kMaxCols;
                float part[4] = {0.f, 0.f, 0.f, 0.f};
                uint32_t r[2][16];
                tmem_ld16(src, r[0]);
                for (int n = 0; n < count; n += 32) {
                    tc_wait_ld();
                    if (n + 16 < count) tmem_ld16(src + n + 16, r[1]);
                    if (mask || n >= whole) add_columns<CAP, true>(part, r[0], tab, n, j, a);
                    else add_columns<CAP, false>(part, r[0], tab, n, j, a);
                    if (n + 16 >= count) break;
                    tc_wait_ld();
                    if (n + 32 < count) tmem_ld16(src + n + 32, r[0]);
                    if (mask || n + 16 >= whole) add_columns<CAP, true>(part, r[1], tab, n + 16, j, a);
                    else add_columns<CAP, false>(part, r[1], tab, n + 16, j, a);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_empty[group]);
                // sum + lost += part (a sum with its rounding error kept)
                const float more = (part[0] + part[1]) + (part[2] + part[3]) + lost, now = sum + more;
                lost = more - (now - sum);
                sum = now;
            }
            if (!ok) break;
            if (a.keys_held) {  // the second epilogue's share of the item, through shared memory
                if (group == 1) {
                    if (!(ok = wait_warp(&x_empty[quarter], (items & 1) ^ 1))) break;
                    passed[row] = sum + lost;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&x_full[quarter]);
                } else {
                    if (!(ok = wait_warp(&x_full[quarter], items & 1))) break;
                    sum += passed[row] + lost;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&x_empty[quarter]);
                }
            }
            if (writes && j < it.len) *dst = was + sum;
        }
    }
    __syncthreads();
    if (tid == 0 && *abort_flag) report_status(a.status, kErrTimeout);
    if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

// ---------------------------------------------------------------------------------- fp32
constexpr int kF32Keys = 64, kF32Depth = 32, kF32Threads = 128;

// One CTA: 64 keys of one (sequence, KV head) over its columns, COLS at once.  Thread (x, y) takes
// keys 4 x .. 4 x + 3 and columns y, y + 8, ...
template <int COLS, bool CAP>
__global__ void __launch_bounds__(kF32Threads) key_weights_f32_kernel(const KeyWeightsArgs a) {
    constexpr int kPer = COLS / 8;
    __shared__ float sK[kF32Depth][kF32Keys + 4], sQ[kF32Depth][COLS + 1];
    __shared__ float lse2[COLS];
    __shared__ int hi[COLS], lo[COLS];
    const int tid = threadIdx.x, x = tid / 8, y = tid % 8;
    const int b = blockIdx.y / a.n_kv_heads, hk = blockIdx.y % a.n_kv_heads, G = a.n_heads / a.n_kv_heads, D = a.head_dim;
    const int raw = a.kv_lens[b], first = (int)blockIdx.x * kF32Keys;
    if (raw < 0 || raw > a.max_kv_len) {
        if (blockIdx.x == 0 && hk == 0 && tid == 0) report_status(a.status, kErrBounds);
        return;
    }
    if (first >= raw) return;
    const int last = min(first + kF32Keys, raw) - 1;
    const int64_t off = (int64_t)raw - a.n_q;
    int64_t i0 = max((int64_t)0, -off), i1 = a.n_q - 1;
    if (a.causal) i0 = max(i0, first - off);
    if (a.window > 0) i1 = min(i1, (int64_t)last + a.window - 1 - off);
    if (i0 > i1) return;
    const float *kb = static_cast<const float *>(a.k) + (int64_t)b * a.k_seq + (int64_t)hk * a.k_head;
    float sum[4] = {0.f, 0.f, 0.f, 0.f}, lost[4] = {0.f, 0.f, 0.f, 0.f};
    for (int64_t c0 = i0 * G; c0 < (i1 + 1) * G; c0 += COLS) {
        __syncthreads();  // the table is free
        for (int c = tid; c < COLS; c += kF32Threads) {
            const int64_t col = c0 + c;
            lse2[c] = INFINITY, hi[c] = -1, lo[c] = -1;
            if (col < (i1 + 1) * G) {
                const int64_t i = col / G, pos = off + i;
                const float l = a.lse[((int64_t)b * a.n_q + i) * a.n_heads + hk * G + col % G];
                if (l != -INFINITY) {
                    lse2[c] = l * 1.4426950408889634f;
                    hi[c] = a.causal ? (int)pos : 0x7fffffff;
                    lo[c] = a.window > 0 ? (int)pos - a.window : -1;
                }
            }
        }
        float s[4][kPer];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int c = 0; c < kPer; ++c) s[k][c] = 0.f;
        for (int d0 = 0; d0 < D; d0 += kF32Depth) {
            __syncthreads();
            for (int e = tid; e < kF32Keys * kF32Depth; e += kF32Threads) {
                const int d = e % kF32Depth, r = e / kF32Depth;
                sK[d][r] = d0 + d < D && first + r <= last ? kb[(int64_t)(first + r) * a.k_row + d0 + d] : 0.f;
            }
            for (int e = tid; e < COLS * kF32Depth; e += kF32Threads) {
                const int d = e % kF32Depth, c = e / kF32Depth;
                const int64_t col = c0 + c, i = col / G;
                sQ[d][c] = d0 + d < D && col < (i1 + 1) * G
                               ? static_cast<const float *>(a.q)[((int64_t)b * a.n_q + i) * a.q_rs + (int64_t)(hk * G + col % G) * D + d0 + d]
                               : 0.f;
            }
            __syncthreads();
#pragma unroll 8
            for (int d = 0; d < kF32Depth; ++d) {
                const float4 k4 = *reinterpret_cast<const float4 *>(&sK[d][4 * x]);
#pragma unroll
                for (int c = 0; c < kPer; ++c) {
                    const float q = sQ[d][y + 8 * c];
                    s[0][c] = fmaf(k4.x, q, s[0][c]);
                    s[1][c] = fmaf(k4.y, q, s[1][c]);
                    s[2][c] = fmaf(k4.z, q, s[2][c]);
                    s[3][c] = fmaf(k4.w, q, s[3][c]);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float part = 0.f;
            const int j = first + 4 * x + k;
#pragma unroll
            for (int c = 0; c < kPer; ++c) {
                const int n = y + 8 * c;
                const float v = CAP ? a.cap_log2 * tanhf(s[k][c] * a.raw_over_cap) - lse2[n] : fmaf(s[k][c], a.scale_log2, -lse2[n]);
                part += j <= hi[n] && j > lo[n] ? fast_exp2(v) : 0.f;
            }
            const float more = part + lost[k], now = sum[k] + more;
            lost[k] = more - (now - sum[k]);
            sum[k] = now;
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float v = sum[k] + lost[k];
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        const int j = first + 4 * x + k;
        if (y == 0 && j <= last) a.weights[(int64_t)b * a.w_seq + (int64_t)hk * a.w_head + j] += v;
    }
}

template <int D>
int held_cols() { return KwCfg<D>::kHeldCols; }

template <int D, bool CAP>
cudaError_t launch_tc(const KeyWeightsArgs &a, int grid, cudaStream_t s) {
    using C = KwCfg<D>;
    const cudaError_t e = cudaFuncSetAttribute(key_weights_kernel<D, CAP>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    key_weights_kernel<D, CAP><<<grid, kTcThreads, C::kSmem, s>>>(a);
    return cudaGetLastError();
}
template <int D>
cudaError_t launch_d(const KeyWeightsArgs &a, int grid, cudaStream_t s) {
    return a.cap_log2 > 0.f ? launch_tc<D, true>(a, grid, s) : launch_tc<D, false>(a, grid, s);
}

}  // namespace

bool plan_key_weights(int batch, int n_q, int n_heads, int n_kv_heads, int head_dim, int max_kv_len, int num_sms,
                      KeyWeightsPlan *p) {
    const int G = n_heads / n_kv_heads;
    int most = 0;
    switch (head_dim) {
        case 64: most = held_cols<64>(); break;
        case 80: most = held_cols<80>(); break;
        case 128: most = held_cols<128>(); break;
        case 256: most = held_cols<256>(); break;
        case 512: most = held_cols<512>(); break;
        default: return false;
    }
    const int64_t cols = (int64_t)n_q * G;
    p->keys_held = cols > most;
    if (!p->keys_held) {
        p->heads_per = G;
        p->rows_per = n_q;
        p->head_blocks = 1;
    } else if (G <= kStreamCols) {
        p->heads_per = G;
        p->rows_per = std::min(n_q, kStreamCols / G);
        p->head_blocks = 1;
    } else {
        p->heads_per = kStreamCols;
        p->rows_per = 1;
        p->head_blocks = (G + kStreamCols - 1) / kStreamCols;
    }
    p->n_cols = (p->rows_per * p->heads_per + 15) / 16 * 16;
    const int64_t items = ((int64_t)max_kv_len + kKeysTile - 1) / kKeysTile * batch * n_kv_heads;
    p->slots = items;
    p->grid = (int)std::min<int64_t>(num_sms, std::max<int64_t>(items, 1));
    return true;
}

cudaError_t launch_key_weights(const KeyWeightsArgs &a, int grid, cudaStream_t s) {
    switch (a.head_dim) {
        case 64: return launch_d<64>(a, grid, s);
        case 80: return launch_d<80>(a, grid, s);
        case 128: return launch_d<128>(a, grid, s);
        case 256: return launch_d<256>(a, grid, s);
        case 512: return launch_d<512>(a, grid, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_key_weights_f32(const KeyWeightsArgs &a, cudaStream_t s) {
    // (one block of nothing still sees the lengths)
    const dim3 grid((unsigned)((std::max<int64_t>(a.max_kv_len, 1) + kF32Keys - 1) / kF32Keys), (unsigned)(a.batch * a.n_kv_heads));
    const bool cap = a.cap_log2 > 0.f;
    if ((int64_t)a.n_q * (a.n_heads / a.n_kv_heads) <= 8) {
        if (cap) key_weights_f32_kernel<8, true><<<grid, kF32Threads, 0, s>>>(a);
        else key_weights_f32_kernel<8, false><<<grid, kF32Threads, 0, s>>>(a);
    } else {
        if (cap) key_weights_f32_kernel<64, true><<<grid, kF32Threads, 0, s>>>(a);
        else key_weights_f32_kernel<64, false><<<grid, kF32Threads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace lat
