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
//    (Tiles of 256 columns where there are as many: an MMA of 128 x 128 x 16 reads both operands at
//    what shared memory gives, one of twice the columns three quarters of it.)
//  * Roles: epilogue warps in quartets (a warp can read the quarter of tensor memory's lanes that
//    its number says), a warp that issues the copies, one that issues the MMAs, two that prepare
//    the columns' log-sum-exps and ranges of keys.  S has four buffers of 128 columns in tensor
//    memory; the quartets take tiles of S in turn, each whole, so that its waits are few.  Where a
//    key tile has several tiles of S, the quartets' sums meet in shared memory at its end.  Where a range
//    cuts a tile, pairs are masked one by one.
//  * What a role does for every tile is kept short (a wait that need not wait costs a thread 100
//    to 200 cycles): walks go by runs of tiles, tables come with the tile of S they belong to, and
//    a key's sum goes to memory as a reduction that nothing waits for.
//  * A pair costs half an FMA and half an addition (f32x2) and one exponential.  A thread adds a
//    tile's columns in four sums and those to its total with a compensation, so prompts of many
//    thousand rows lose nothing.
//  * Waits are bounded; on expiry the CTA records LAT_ERR_TIMEOUT, drains and quits.
// What bounds it: HBM (keys once) for few columns; for many the tensor pipe and the exponentials,
// 128 N D 2 flops against 128 N of them.
//
// fp32 (key_weights_f32_kernel): fp32 products by FMA, 64 keys x 32 or 64 columns a step, a thread 4
// x 4 or 8 of them; the next 32 channels come while 32 are used.  Bound by its FMAs, or by their
// chain where keys are few: then a cluster shares the columns (one sequence of 200 keys and rows, 12
// heads over one: 231 -> 30 us in eight CTAs).  Up to eight
// columns (a decode step) go to key_weights_few_kernel, whose keys do not pass through shared
// memory (2 x 40000 keys, 24 heads over 8, head_dim 128: 75.7 -> 47.6 us, 3.5 TB/s; 32 caches of up
// to 4096, 12 heads over 4, head_dim 64: 35.8 -> 26.5).  It is bound by what a key costs beside its
// products: 31 exchanges for 32 sums, each two selections, a shuffle and an addition.
#include <math.h>

#include <algorithm>

#include "cache_kernels.h"
#include "device_common.cuh"
#include "f32x2.cuh"
#include "score_cap.cuh"
#include "tc_desc.cuh"

namespace lat {

namespace {

constexpr int kKeysTile = 128;
constexpr int kMaxCols = 256;                     // columns of a tile
constexpr int kQuartets = 2, kEpilogue = 4 * kQuartets;  // of epilogue warps; those
constexpr int kMoreWarps = 4;                     // behind them: copies, MMAs, two of tables
constexpr int kThreads = 32 * (kEpilogue + kMoreWarps);
constexpr int kTables = 4;
constexpr int kPlaces = 4;                        // key tiles whose sums can be under way at once
constexpr int kSBufs = 4, kSCols = 128;           // tiles of S in tensor memory
constexpr uint32_t kTmemCols = kSBufs * kSCols;
constexpr int kMaxStages = 8, kMaxHeld = 8;

template <int D>
struct KwCfg {
    static constexpr int kChunks = (D + 63) / 64;           // 64-channel chunks of a row
    static constexpr int kSteps = (D + 15) / 16;            // MMAs of a tile
    static constexpr int kStageChunks = D == 64 ? 1 : 2;    // chunks of keys in a ring stage, 16 KB each
    static constexpr int kStageBytes = kStageChunks * 16384;
    // The operand that stays has up to 64 KB (head_dim 512: 128 KB): up to 256 (head_dim 256, 512: 128)
    // columns, or 128 keys.  What it leaves of kTiles is the ring's.
    static constexpr int kHeldBytes = D == 512 ? 131072 : 65536;
    static constexpr int kHeldCols = kHeldBytes / (kChunks * 128) < kMaxCols ? kHeldBytes / (kChunks * 128) : kMaxCols;
    static constexpr int kManyHeldBytes = 32768;
    static constexpr int kTiles = 196608;
    static constexpr int kTableBytes = kTables * (3 * kMaxCols + 4) * 4;
    static constexpr int kPassed = kPlaces * kKeysTile * 4;  // [key tile % kPlaces][key] sums
    static constexpr int kBarBytes = 1024;
    static constexpr int kSmem = kTiles + kTableBytes + kPassed + kBarBytes;
    static_assert(kSmem <= 232448, "shared memory budget");
};

// the columns of a tile: e^{s - lse} = 2^(s' - lse2), and the keys lo < j <= hi that a column sees
struct Table {
    float minus_lse2[kMaxCols];
    int hi[kMaxCols], lo[kMaxCols];
    int min_hi, max_lo, count, pad;  // over the columns there are
};

// tiles one after another that share the operand that stays
struct Run {
    int b, hk, len;
    int t, n;   // queries held: key tiles t .. t + n - 1; keys held: key tile t and n tiles of columns,
    int64_t x;  // x .. x + n - 1
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

// The CTA's runs.  Queries held: a share of all (b, hk, t) in this order; keys held: every grid-th
// of all (t, b, hk), forwards and backwards in turn.
struct Walker {
    const KeyWeightsArgs &a;
    int64_t pos, end;  // next tile, and behind the last; or the round
    int64_t base;      // queries held: where sequence b's tiles begin
    int b;
    int of, len;       // queries held: the sequence whose length is at hand, and that
    int2 seen;

    __device__ bool next(Run &r) { return a.keys_held ? next_dealt(r) : next_shared(r); }
    __device__ bool next_shared(Run &r) {
        if (pos >= end) return false;
        for (;; ++b) {
            if (b != of) of = b, len = length_of(a, b), seen = tiles_seen(a, len);
            r.len = len;
            const int n = seen.y - seen.x;
            const int64_t all = (int64_t)n * a.n_kv_heads;
            if (pos >= base + all) {
                base += all;
                continue;
            }
            const uint32_t at = (uint32_t)(pos - base);  // (items are fewer than 2^31)
            r.b = b;
            r.hk = (int)(at / (uint32_t)n);
            r.t = seen.x + (int)(at % (uint32_t)n);
            r.n = (int)min((int64_t)(seen.y - r.t), end - pos);
            r.x = 0;
            pos += r.n;
            return true;
        }
    }
    __device__ bool next_dealt(Run &r) {
        const int64_t per = (int64_t)a.batch * a.n_kv_heads;
        for (;; ++pos) {
            const int64_t x = pos * gridDim.x + ((pos & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
            if (pos * gridDim.x >= end) return false;
            if (x >= end) continue;
            r.t = (int)(x / per);
            const int rem = (int)(x - r.t * per);
            r.b = rem / a.n_kv_heads;
            r.hk = rem - r.b * a.n_kv_heads;
            r.len = length_of(a, r.b);
            const int2 seen = tiles_seen(a, r.len);
            if (r.t < seen.x || r.t >= seen.y) continue;
            // rows that see a key of the tile
            const int64_t off = (int64_t)r.len - a.n_q, first = (int64_t)r.t * kKeysTile;
            const int64_t last = min(first + kKeysTile, (int64_t)r.len) - 1;
            int64_t i0 = max((int64_t)0, -off), i1 = a.n_q - 1;
            if (a.causal) i0 = max(i0, first - off);
            if (a.window > 0) i1 = min(i1, last + a.window - 1 - off);
            if (i0 > i1) continue;
            r.x = i0 / a.rows_per * a.head_blocks;
            r.n = (int)((i1 / a.rows_per + 1) * a.head_blocks - r.x);
            ++pos;
            return true;
        }
    }
};

// sums over 16 columns (the table's from n on) of 2^(s' - lse2), the scores as they came out of the
// MMA; two a sum
template <bool CAP, bool MASK>
__device__ __forceinline__ void add_columns(uint64_t (&sum)[2], const uint32_t (&r)[16], const Table &tab, int n, int j,
                                            const KeyWeightsArgs &a) {
    uint64_t x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = pair_of(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1]));
    // A capped score is cap * y * f(y^2), y the score over the cap, f(z) = tanh(sqrt z) / sqrt z.  Most
    // lie well below the cap, where f is a polynomial through Chebyshev's nodes of [0, 0.0225] (to z^2,
    // within 4e-8) or [0, 0.09] (to z^3, 2e-8).  Which form serves is decided by the pairs
    // that count: what else lies in the tile must not show in a key's bits.
    uint64_t f[8];
    uint32_t seen = 0;  // which columns see the key
    if constexpr (CAP && MASK) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int4 hi = *reinterpret_cast<const int4 *>(tab.hi + n + 4 * q);
            const int4 lo = *reinterpret_cast<const int4 *>(tab.lo + n + 4 * q);
            seen |= (j <= hi.x && j > lo.x ? 1u << 4 * q : 0u) | (j <= hi.y && j > lo.y ? 2u << 4 * q : 0u) |
                    (j <= hi.z && j > lo.z ? 4u << 4 * q : 0u) | (j <= hi.w && j > lo.w ? 8u << 4 * q : 0u);
        }
    }
    if constexpr (CAP) {
        float most = 0.f;
        uint64_t z[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            x[k] = mul2(x[k], twice(a.raw_over_cap));
            z[k] = mul2(x[k], x[k]);
            const float2 y = halves_of(z[k]);
            if constexpr (MASK) most = fmaxf(most, fmaxf(seen & 1u << 2 * k ? y.x : 0.f, seen & 2u << 2 * k ? y.y : 0.f));
            else most = fmaxf(most, fmaxf(y.x, y.y));
        }
        const float c = a.cap_log2;
        if (!__any_sync(0xffffffffu, !(most < 0.0225f))) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                f[k] = fma2(z[k], fma2(z[k], twice(c * 0.13153041899204254f), twice(c * -0.33331817388534546f)), twice(c));
        } else if (!__any_sync(0xffffffffu, !(most < 0.09f))) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint64_t t = fma2(z[k], twice(c * -0.05022099241614342f), twice(c * 0.13312578201293945f));
                f[k] = fma2(z[k], fma2(z[k], t, twice(c * -0.33332961797714233f)), twice(c));
            }
        } else {  // (scores as they are, for the sum below)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 y = halves_of(x[k]);
                x[k] = pair_of(capped_score_close(y.x, c), capped_score_close(y.y, c));
                f[k] = twice(1.f);
            }
        }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float4 l = *reinterpret_cast<const float4 *>(tab.minus_lse2 + n + 4 * q);
        const uint64_t ls[2] = {pair_of(l.x, l.y), pair_of(l.z, l.w)};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint64_t y = fma2(x[2 * q + k], CAP ? f[2 * q + k] : twice(a.scale_log2), ls[k]);
            float2 p = halves_of(y);
            p.x = fast_exp2(p.x), p.y = fast_exp2(p.y);
            if constexpr (CAP && MASK) {
                p.x = seen & 1u << (4 * q + 2 * k) ? p.x : 0.f;
                p.y = seen & 2u << (4 * q + 2 * k) ? p.y : 0.f;
            } else if constexpr (MASK) {
                const int2 hi = *reinterpret_cast<const int2 *>(tab.hi + n + 4 * q + 2 * k);
                const int2 lo = *reinterpret_cast<const int2 *>(tab.lo + n + 4 * q + 2 * k);
                p.x = j <= hi.x && j > lo.x ? p.x : 0.f;
                p.y = j <= hi.y && j > lo.y ? p.y : 0.f;
            }
            sum[k] = add2(sum[k], pair_of(p.x, p.y));
        }
    }
}

template <int D, bool CAP>
__global__ void __launch_bounds__(kThreads, 1) key_weights_kernel(const __grid_constant__ KeyWeightsArgs a) {
    using C = KwCfg<D>;
    extern __shared__ __align__(1024) unsigned char smem[];      // (an aligned-up pointer would load as generic)
    Table *tables = reinterpret_cast<Table *>(smem + C::kTiles);  // [kTables]
    float *passed = reinterpret_cast<float *>(tables + kTables);  // [key tile % kPlaces][key]
    uint64_t *bars = reinterpret_cast<uint64_t *>(passed + kPlaces * kKeysTile);
    uint64_t *ring_full = bars, *ring_empty = bars + 8;          // [n_stages]
    uint64_t *held_full = bars + 16, *held_empty = bars + 24;    // [n_held]
    uint64_t *s_full = bars + 32, *s_empty = bars + 36;          // [4]
    uint64_t *tab_full = bars + 40, *tab_empty = tab_full + kTables;
    uint64_t *x_full = tab_empty + kTables;                      // [key tile % kPlaces][quarter of the lanes]
    uint64_t *bar_done = x_full + 4 * kPlaces;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar_done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int64_t *start = reinterpret_cast<int64_t *>(bar_done + 2);  // share: base, b
    int *scan = reinterpret_cast<int *>(bar_done + 4);           // a warp each
    static_assert(sizeof(Table) * kTables == C::kTableBytes && kTables >= kSBufs &&
                      (44 + 2 * kTables + 4 * kPlaces) * 8 + kThreads / 32 * 4 <= C::kBarBytes,
                  "shared memory layout");
    if (smem_u32(smem) & 1023) {  // (swizzled operands need it; it is where dynamic shared memory begins)
        if (threadIdx.x == 0) report_status(a.status, kErrCuda);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // what takes a round trip first: the first of this thread's lengths, the tensor maps (there are none
    // for caches that hold nothing)
    const int per_thread = (a.batch + kThreads - 1) / kThreads;
    const int b_lo = min(a.batch, tid * per_thread), b_hi = min(a.batch, b_lo + per_thread);
    const int len_lo = b_lo < b_hi ? a.kv_lens[b_lo] : 0;
    if (tid == 0 && a.max_kv_len > 0) tma_prefetch_desc(&a.tm_q), tma_prefetch_desc(&a.tm_k);
    const int halves = a.n_cols > kSCols ? 2 : 1;                // tiles of S of a column tile (queries held)
    // bytes of a chunk of the tile of queries and of keys; how many operands there is room to hold,
    // and stages behind them
    const int q_rows = a.rows_per * a.heads_per;                 // columns that a copy brings
    const int q_chunk = a.n_cols * 128;                          // where its chunks lie apart
    const int held_bytes = C::kChunks * (a.keys_held ? 16384 : q_chunk);
    // (two where there is room, more while they are small: short sequences are over before the next
    // one's queries have come.  32 sequences of 1 to 4096 keys, one row: two 36.2 us, eight 32.2)
    int held_log2 = 2 * held_bytes <= C::kHeldBytes ? 1 : 0;
    while (!a.keys_held && (2 << held_log2) <= kMaxHeld && (2 << held_log2) * held_bytes <= C::kManyHeldBytes) ++held_log2;
    const unsigned n_held = 1u << held_log2;
    unsigned char *held = smem, *ring = held + n_held * held_bytes;
    const int stage_bytes = a.keys_held ? q_chunk : C::kStageBytes;  // of queries, one chunk
    const int stage_chunks = a.keys_held ? 1 : C::kStageChunks, per_tile = C::kChunks / stage_chunks;
    const unsigned n_stages = min(kMaxStages, (C::kTiles - (int)n_held * held_bytes) / stage_bytes);
    const int G = a.n_heads / a.n_kv_heads;
    const uint64_t deadline = globaltimer_ns() + a.timeout_ns;
    if (tid < 32) {  // barriers, a few a lane
        auto init = [&](uint64_t *first, int n, int count) {
            if (lane < n) mbar_init(first + lane, count);
        };
        init(ring_full, 2 * kMaxStages + 2 * kMaxHeld, 1);  // ring and held
        init(s_full, kSBufs, a.keys_held ? 2 : 1);  // keys held: full when its MMAs are done and its table is there
        init(s_empty, kSBufs, 4 * halves);
        init(tab_full, kTables, 1);
        init(tab_empty, kTables, kEpilogue);
        init(x_full, 4 * kPlaces, 1);
        init(bar_done, 1, 1);
        if (lane == 0) *abort_flag = 0, start[0] = 0, start[1] = a.batch;
        fence_mbarrier_init();
    }
    if (warp == kEpilogue + 1) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    // ---- this CTA's share: per-thread sums over a slice of the sequences, then a scan ----------
    // (item counts stay below 2^31)
    int mine = 0;
    for (int b = b_lo; b < b_hi; ++b) {
        const int n = b == b_lo ? len_lo : a.kv_lens[b];
        const bool bad = n < 0 || n > a.max_kv_len;
        if (blockIdx.x == 0 && bad) report_status(a.status, kErrBounds);
        const int2 seen = tiles_seen(a, bad ? 0 : n);
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
    const int of_warp = lane < kThreads / 32 ? scan[lane] : 0;
    const int total = __reduce_add_sync(0xffffffffu, of_warp);
    const int before = incl - mine + __reduce_add_sync(0xffffffffu, lane < warp ? of_warp : 0);
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
    Walker walk{a, r0, r1, start[0], (int)start[1], -1};
    auto wait = [&](uint64_t *bar, uint32_t parity) { return mbar_wait_bounded(bar, parity, abort_flag, deadline); };

    if (warp == kEpilogue) {
        if (lane == 0) {
            unsigned g = 0, h = 0, s = 0, turn = 0;  // stages and held operands issued; place in the ring, times round it
            bool ok = true;
            // chunks [c0, c1) of key tile t, and of the columns of row block rb and head block hb
            auto keys = [&](unsigned char *to, uint64_t *bar, const Run &r, int t, int c0, int c1) {
                for (int c = c0; c < c1; ++c)
                    tma_load_4d(to + (c - c0) * 16384, &a.tm_k, bar, c * 64, r.hk, t * kKeysTile, r.b);
            };
            auto queries = [&](unsigned char *to, uint64_t *bar, const Run &r, int rb, int hb, int c0, int c1) {
                for (int c = c0; c < c1; ++c)
                    tma_load_4d(to + (c - c0) * q_chunk, &a.tm_q, bar, c * 64, r.hk * G + hb * a.heads_per, rb * a.rows_per, r.b);
            };
            for (Run r; ok && walk.next(r); ++h) {
                const unsigned y = h & (n_held - 1);
                if (!(ok = wait(&held_empty[y], ((h >> held_log2) & 1) ^ 1))) break;
                mbar_arrive_expect_tx(&held_full[y], C::kChunks * (a.keys_held ? 16384 : q_rows * 128));
                if (a.keys_held) keys(held + y * held_bytes, &held_full[y], r, r.t, 0, C::kChunks);
                else queries(held + y * held_bytes, &held_full[y], r, 0, 0, 0, C::kChunks);
                int rb = (int)(r.x / a.head_blocks), hb = (int)(r.x - (int64_t)rb * a.head_blocks);
                for (int i = 0; ok && i < r.n; ++i) {
                    for (int p = 0; p < per_tile; ++p, ++g) {
                        if (turn > 0 && !(ok = wait(&ring_empty[s], (turn & 1) ^ 1))) break;
                        if (!a.test_skip_load || g > 0) {  // (test hook: the first never comes)
                            mbar_arrive_expect_tx(&ring_full[s], a.keys_held ? q_rows * 128 : C::kStageBytes);
                            if (a.keys_held) queries(ring + s * stage_bytes, &ring_full[s], r, rb, hb, p, p + 1);
                            else keys(ring + s * stage_bytes, &ring_full[s], r, r.t + i, p * C::kStageChunks, (p + 1) * C::kStageChunks);
                        }
                        if (++s == n_stages) s = 0, ++turn;
                    }
                    if (++hb == a.head_blocks) hb = 0, ++rb;
                }
            }
            // every copy lands before the CTA leaves: slot s last held the largest fill s + k * slots
            const uint64_t until = globaltimer_ns() + 100000000ull;
            volatile int no_abort = 0;
            for (unsigned x = 0; x < n_stages && x < g; ++x) {
                const unsigned last = x + (g - 1 - x) / n_stages * n_stages;
                if (!(a.test_skip_load && last == 0)) mbar_wait_bounded(&ring_full[x], (last / n_stages) & 1, &no_abort, until);
            }
            for (unsigned x = 0; x < n_held && x < h; ++x) {
                const unsigned last = x + (h - 1 - x) / n_held * n_held;
                mbar_wait_bounded(&held_full[x], (last / n_held) & 1, &no_abort, until);
            }
        }
        __syncwarp();
    } else if (warp == kEpilogue + 1) {
        if (lane == 0) {
            // N is the whole tile of columns: its two tiles of S lie side by side
            const uint32_t idesc = instr_desc(kKeysTile, a.n_cols, false);
            const uint64_t d_ring = sw128_desc(smem_u32(ring)), d_held = sw128_desc(smem_u32(held));
            // a chunk of keys is 16 KB wherever it lies
            const uint64_t q_step = q_chunk >> 4, part = a.keys_held ? 1024 : C::kStageChunks * q_step;
            unsigned h = 0, step = 0, s = 0, turn = 0;  // held operands, tiles of S; place in the ring, times round it
            bool ok = true;
            for (Run r; ok && walk.next(r); ++h) {
                const unsigned y = h & (n_held - 1);
                if (!(ok = wait(&held_full[y], (h >> held_log2) & 1))) break;
                const uint64_t kept = d_held + (uint64_t)((y * held_bytes) >> 4);
                for (int i = 0; ok && i < r.n; ++i, step += halves) {
                    const unsigned buf = step % kSBufs;  // (two tiles of S lie side by side and go by the first's barriers)
                    if (step >= kSBufs && !(ok = wait(&s_empty[buf], ((step / kSBufs) & 1) ^ 1))) break;
                    const uint32_t d = tmem + buf * kSCols;
                    for (int p = 0; p < per_tile; ++p) {
                        if (!(ok = wait(&ring_full[s], turn & 1))) break;
                        tc_fence_after();
                        const uint64_t here = d_ring + (uint64_t)((s * stage_bytes) >> 4), there = kept + p * part;
                        const uint64_t dk = a.keys_held ? there : here, dq = a.keys_held ? here : there;
#pragma unroll
                        for (int c = 0; c < C::kStageChunks; ++c) {
                            if (c >= stage_chunks) break;
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (D % 64 == 0 || (p * stage_chunks + c) * 4 + k < C::kSteps)
                                    tc_mma_ss(d, dk + (uint64_t)((c * 16384 + k * 32) >> 4), dq + c * q_step + (uint64_t)(k * 32 >> 4),
                                              idesc, p > 0 || c > 0 || k > 0);
                        }
                        tc_commit(&ring_empty[s]);
                        if (++s == n_stages) s = 0, ++turn;
                    }
                    if (ok) tc_commit(&s_full[buf]);
                }
                tc_commit(&held_empty[y]);
            }
            // all MMAs finish before tensor memory is freed
            tc_commit(bar_done);
            volatile int no_abort = 0;
            mbar_wait_bounded(bar_done, 0, &no_abort, globaltimer_ns() + 100000000ull);
        }
        __syncwarp();
    } else if (warp >= kEpilogue + 2) {
        // ---- tables.  Queries held: one a run, the warps in turn.  Keys held: one a tile of columns,
        // the warps in turn, in the place of its tile of S; the next one's log-sum-exps are on their way
        // while one is filled.  Lane i has columns i, i + 32, ...: rows and heads that do not change.
        constexpr int kMine = kMaxCols / 32;
        const int odd = warp - kEpilogue - 2;
        int col_row[kMine], col_at[kMine];
#pragma unroll
        for (int e = 0; e < kMine; ++e) {
            const uint32_t i = lane + 32 * e;
            col_row[e] = (int)a.by_heads_per.div(i);
            col_at[e] = col_row[e] * a.n_heads + (int)i - col_row[e] * a.heads_per;
        }
        struct Place {
            int rb, hb, count;
        };
        auto place_of = [&](int64_t x) {  // (one block of heads, or one row a tile: the columns there are come first)
            Place p;
            p.rb = (int)(x / a.head_blocks), p.hb = (int)(x - (int64_t)p.rb * a.head_blocks);
            p.count = min(a.rows_per, a.n_q - p.rb * a.rows_per) * min(a.heads_per, G - p.hb * a.heads_per);
            return p;
        };
        float l[kMine];
        auto ask = [&](const Run &r, const Place &p) {
            const float *src = a.lse + ((int64_t)r.b * a.n_q + p.rb * a.rows_per) * a.n_heads + r.hk * G + p.hb * a.heads_per;
#pragma unroll
            for (int e = 0; e < kMine; ++e) {
                if (32 * e >= a.n_cols) break;
                l[e] = lane + 32 * e < p.count ? __ldg(src + col_at[e]) : -INFINITY;
            }
        };
        auto fill = [&](Table &tab, const Run &r, const Place &p) {
            const int pos0 = r.len - a.n_q + p.rb * a.rows_per;
            int min_hi = 0x7fffffff, max_lo = -1;
#pragma unroll
            for (int e = 0; e < kMine; ++e) {
                const int i = lane + 32 * e, pos = pos0 + col_row[e];
                if (32 * e >= a.n_cols) break;
                int hi = -1, lo = -1;
                if (i < p.count) {
                    if (pos >= 0 && l[e] != -INFINITY) {  // (else the row sees nothing)
                        hi = a.causal ? pos : CAP ? r.len - 1 : 0x7fffffff;
                        lo = a.window > 0 ? pos - a.window : -1;
                    }
                    min_hi = min(min_hi, hi);
                    max_lo = max(max_lo, lo);
                }
                tab.minus_lse2[i] = l[e] == -INFINITY ? -INFINITY : l[e] * -1.4426950408889634f;
                tab.hi[i] = hi, tab.lo[i] = lo;
            }
            min_hi = __reduce_min_sync(0xffffffffu, min_hi);
            max_lo = __reduce_max_sync(0xffffffffu, max_lo);
            if (lane == 0) tab.min_hi = min_hi, tab.max_lo = max_lo, tab.count = p.count;
            __syncwarp();
        };
        auto wait_warp = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
        unsigned n = 0;  // tables before this run's
        bool ok = true;
        if (!a.keys_held) {
            // this warp's runs, the next one's log-sum-exps on their way while one is filled
            const Place p = place_of(0);
            Run r;
            bool more = walk.next(r) && (odd == 0 || walk.next(r));
            n = odd;
            while (more) {
                ask(r, p);
                Run next = r;
                more = walk.next(next) && walk.next(next);
                const unsigned u = n % kTables;
                if (!(ok = wait_warp(&tab_empty[u], ((n / kTables) & 1) ^ 1))) break;
                fill(tables[u], r, p);
                if (lane == 0) mbar_arrive(&tab_full[u]);
                r = next;
                n += 2;
            }
        }
        for (Run r; a.keys_held && ok && walk.next(r);) {
            int i = (n & 1) == (unsigned)odd ? 0 : 1;  // this warp's first of the run
            Place p = place_of(r.x + i);
            if (i < r.n) ask(r, p);
            for (; i < r.n; i += 2) {
                const unsigned k = 2 * (n + i), u = k % kSBufs;  // its first tile of S
                if (k >= kSBufs && !(ok = wait_warp(&s_empty[u], ((k / kSBufs) & 1) ^ 1))) break;
                fill(tables[u], r, p);
                if (lane == 0) mbar_arrive(&s_full[u]);
                if (i + 2 < r.n) {
                    p = place_of(r.x + i + 2);
                    ask(r, p);
                }
            }
            n += r.n;
        }
    } else {
        // ---- epilogues: thread = key ----------------------------------------------------------
        const int quartet = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        auto wait_warp = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
        // the sum over the tile of S of that number, its columns the table's from `off` on; false: a wait
        // ran out
        auto take = [&](unsigned step, const Table &tab, int off, int first, int last, float &total) {
            const unsigned buf = step % kSBufs, bar = buf & -halves;
            if (!wait_warp(&s_full[bar], (step / kSBufs) & 1)) return false;
            tc_fence_after();
            const int n1 = max(1, min(tab.count - off, kSCols)), j = first + row;  // (one that is not there is masked)
            // (capped, keys that are not there must be known, so that they do not vote)
            const bool mask = tab.min_hi < last || tab.max_lo >= first || (CAP && last - first < kKeysTile - 1);
            const uint32_t src = lanes + buf * kSCols;
            uint64_t part[2] = {0, 0};
            auto let_go = [&] {  // S may be written again (with keys held, the table too)
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_empty[bar]);
            };
            // 64 columns at a time where none is masked, so that loads, FMAs and exponentials of many overlap
            // (sixteen at a time by twice the warps with half the registers: 64 rows over four caches 49.3 us,
            // so 44.2; a prompt at head_dim 128 159, so 123)
            if (n1 == kSCols && !mask) {
                uint32_t r[4][16];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) tmem_ld16(src + 64 * h + 16 * q, r[q]);
                    tc_wait_ld();
                    if (h == 1 && !a.keys_held) let_go();
#pragma unroll
                    for (int q = 0; q < 4; ++q) add_columns<CAP, false>(part, r[q], tab, off + 64 * h + 16 * q, j, a);
                }
            } else {
                int n = 0;
                if (!mask && n1 >= 64) {
                    uint32_t r[4][16];
#pragma unroll
                    for (int q = 0; q < 4; ++q) tmem_ld16(src + 16 * q, r[q]);
                    tc_wait_ld();
                    if (n1 == 64 && !a.keys_held) let_go();
#pragma unroll
                    for (int q = 0; q < 4; ++q) add_columns<CAP, false>(part, r[q], tab, off + 16 * q, j, a);
                    n = 64;
                }
                for (; n < n1; n += 16) {
                    uint32_t r[16];
                    tmem_ld16(src + n, r);
                    tc_wait_ld();
                    if (n + 16 >= n1 && !a.keys_held) let_go();
                    if (mask || n + 16 > n1) add_columns<CAP, true>(part, r, tab, off + n, j, a);
                    else add_columns<CAP, false>(part, r, tab, off + n, j, a);
                }
            }
            if (a.keys_held) let_go();
            const float2 p0 = halves_of(part[0]), p1 = halves_of(part[1]);
            total = (p0.x + p0.y) + (p1.x + p1.y);
            return true;
        };
        // The first quartet's sum of key tile number `item`, for the second to add its own.  While that one
        // is still at it, its tiles of S let go, the first gets through two more key tiles at most: the
        // places that it writes to are not this one's.
        auto pass = [&](unsigned item, float sum) {
            const unsigned slot = item % kPlaces;
            passed[slot * kKeysTile + row] = sum;
            __syncwarp();
            if (lane == 0) mbar_arrive(&x_full[slot * 4 + quarter]);
        };
        auto passed_by = [&](unsigned item, float &sum) {
            const unsigned slot = item % kPlaces;
            if (!wait_warp(&x_full[slot * 4 + quarter], (item / kPlaces) & 1)) return false;
            sum += passed[slot * kKeysTile + row];
            return true;
        };
        // (this thread alone has the key: no order of additions comes into it)
        auto give = [&](const Run &r, int t, float sum) {
            const int j = t * kKeysTile + row;
            if (j < r.len && sum != 0.f) atomicAdd(a.weights + (int64_t)r.b * a.w_seq + (int64_t)r.hk * a.w_head + j, sum);
        };
        unsigned step = 0, runs = 0;  // tiles of S, runs before this one
        bool ok = true;
        for (Run r; ok && walk.next(r); ++runs) {
            if (a.keys_held) {  // one key tile; the quartets' tiles of S are the columns' halves
                const int first = r.t * kKeysTile, last = min(first + kKeysTile, r.len) - 1;
                float sum = 0.f, lost = 0.f, part;
                for (int i = 0; i < r.n; ++i, step += 2) {
                    if (!(ok = take(step + quartet, tables[step % kSBufs], quartet * kSCols, first, last, part))) break;
                    // sum + lost += part (a sum with its rounding error kept)
                    const float more = part + lost, now = sum + more;
                    lost = more - (now - sum);
                    sum = now;
                }
                if (!ok) break;
                sum += lost;
                if (quartet == 0) pass(runs, sum);
                else if (!(ok = passed_by(runs, sum))) break;
                else give(r, r.t, sum);
                continue;
            }
            const Table &tab = tables[runs % kTables];
            if (!(ok = wait_warp(&tab_full[runs % kTables], (runs / kTables) & 1))) break;
            const int n = r.n * halves;  // tiles of S
            for (int i = (int)((quartet + step) & 1); i < n; i += 2) {
                const int f = halves == 2 ? quartet : 0, t = r.t + (halves == 2 ? i >> 1 : i);
                const int first = t * kKeysTile, last = min(first + kKeysTile, r.len) - 1;
                const unsigned item = (step + i) >> 1;  // (two halves: step is even)
                float sum;
                if (!(ok = take(step + i, tab, f * kSCols, first, last, sum))) break;
                if (halves == 2 && f == 0) pass(item, sum);
                else if (halves == 2 && !(ok = passed_by(item, sum))) break;
                else give(r, t, sum);
            }
            step += n;
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(&tab_empty[runs % kTables]);
        }
    }
    __syncthreads();
    if (tid == 0 && *abort_flag) report_status(a.status, kErrTimeout);
    if (warp == kEpilogue + 1) tmem_dealloc(tmem, kTmemCols);
}

// ---------------------------------------------------------------------------------- fp32
constexpr int kF32Keys = 64, kF32Depth = 32, kF32Threads = 128;

__device__ __forceinline__ float load_shared_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// A cluster of 2^log2 CTAs (SHARED, else one): 64 keys of one (sequence, KV head) over its columns, COLS at once, a CTA
// its share of them; the first adds the others' sums to its own, in order.  Thread (x, y) takes
// keys 4 x .. 4 x + 3 and columns y, y + 8, ...
template <int COLS, bool CAP, bool SHARED>
__global__ void __launch_bounds__(kF32Threads) key_weights_f32_kernel(const KeyWeightsArgs a, int log2) {
    const int parts_log2 = SHARED ? log2 : 0, parts = 1 << parts_log2;
    constexpr int kPer = COLS / 8, kVecs = kF32Depth / 4;                   // a thread's columns; vectors of a row's 32 channels
    constexpr int kMyK = kF32Keys * kVecs / kF32Threads;                    // a thread's vectors of keys and of queries
    constexpr int kMyQ = COLS * kVecs / kF32Threads;
    __shared__ __align__(16) float sK[kF32Depth][kF32Keys + 4], sQ[kF32Depth][COLS + 4];
    __shared__ float lse2[COLS];
    __shared__ int hi[COLS], lo[COLS];
    __shared__ int64_t q_at[COLS];                                          // where a column's query begins; -1: no column
    const int tid = threadIdx.x, x = tid / 8, y = tid % 8;
    const int b = blockIdx.y / a.n_kv_heads, hk = blockIdx.y % a.n_kv_heads, G = a.n_heads / a.n_kv_heads, D = a.head_dim;
    const int rank = (int)blockIdx.x & (parts - 1);
    const int raw = a.kv_lens[b], first = (int)(blockIdx.x >> parts_log2) * kF32Keys;
    if (raw < 0 || raw > a.max_kv_len) {  // (the whole cluster alike, here and below)
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
    const float *qb = static_cast<const float *>(a.q) + (int64_t)b * a.n_q * a.q_rs + (int64_t)hk * G * D;
    const float *lb = a.lse + (int64_t)b * a.n_q * a.n_heads + hk * G;
    // four channels of a row, from d on
    auto four = [&](const float *p, bool vec) {
        return vec ? __ldg(reinterpret_cast<const float4 *>(p)) : make_float4(__ldg(p), __ldg(p + 1), __ldg(p + 2), __ldg(p + 3));
    };
    float4 kv[kMyK], qv[kMyQ];
    auto ask = [&](int d0) {
#pragma unroll
        for (int e = 0; e < kMyK; ++e) {
            const int v = tid + e * kF32Threads, d = d0 + v % kVecs * 4, r = v / kVecs;
            kv[e] = d < D && first + r <= last ? four(kb + (int64_t)(first + r) * a.k_row + d, a.k_vec) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int e = 0; e < kMyQ; ++e) {
            const int v = tid + e * kF32Threads, d = d0 + v % kVecs * 4, c = v / kVecs;
            const int64_t at = q_at[c];
            qv[e] = d < D && at >= 0 ? four(qb + at + d, a.q_vec) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    float sum[4] = {0.f, 0.f, 0.f, 0.f}, lost[4] = {0.f, 0.f, 0.f, 0.f};
    int64_t c_begin = i0 * G, c_end = (i1 + 1) * G;
    if (SHARED) {  // this CTA's columns, whole steps of them but the last
        const int64_t steps = (c_end - c_begin + COLS - 1) / COLS;
        if (rank + 1 < parts) c_end = c_begin + (steps * (rank + 1) >> parts_log2) * COLS;
        c_begin += (steps * rank >> parts_log2) * COLS;
    }
    for (int64_t c0 = c_begin; c0 < c_end; c0 += COLS) {
        __syncthreads();  // the table is free
        for (int c = tid; c < COLS; c += kF32Threads) {
            lse2[c] = INFINITY, hi[c] = -1, lo[c] = -1, q_at[c] = -1;
            const int64_t col = c0 + c;
            if (col < c_end) {  // (columns are fewer than 2^31)
                const uint32_t i = a.by_heads_per.div((uint32_t)col), g = (uint32_t)col - i * G;
                const int pos = (int)(off + i);
                const float l = lb[(int64_t)i * a.n_heads + g];
                q_at[c] = (int64_t)i * a.q_rs + g * D;
                if (l != -INFINITY) {
                    lse2[c] = l * 1.4426950408889634f;
                    hi[c] = a.causal ? pos : 0x7fffffff;
                    lo[c] = a.window > 0 ? pos - a.window : -1;
                }
            }
        }
        __syncthreads();
        float s[4][kPer];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int c = 0; c < kPer; ++c) s[k][c] = 0.f;
        ask(0);
        for (int d0 = 0; d0 < D; d0 += kF32Depth) {
            if (d0 > 0) __syncthreads();
#pragma unroll
            for (int e = 0; e < kMyK; ++e) {
                const int v = tid + e * kF32Threads, d = v % kVecs * 4, r = v / kVecs;
                sK[d][r] = kv[e].x, sK[d + 1][r] = kv[e].y, sK[d + 2][r] = kv[e].z, sK[d + 3][r] = kv[e].w;
            }
#pragma unroll
            for (int e = 0; e < kMyQ; ++e) {
                const int v = tid + e * kF32Threads, d = v % kVecs * 4, c = v / kVecs;
                sQ[d][c] = qv[e].x, sQ[d + 1][c] = qv[e].y, sQ[d + 2][c] = qv[e].z, sQ[d + 3][c] = qv[e].w;
            }
            __syncthreads();
            if (d0 + kF32Depth < D) ask(d0 + kF32Depth);
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
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[k] = sum[k] + lost[k];
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    }
    __shared__ __align__(16) float mine[kF32Keys];
    if constexpr (SHARED) {
        if (rank > 0 && y == 0) *reinterpret_cast<float4 *>(mine + 4 * x) = make_float4(v[0], v[1], v[2], v[3]);
        cluster_sync_all();
        if (rank == 0 && y == 0)
            for (int p = 1; p < parts; ++p)
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] += load_shared_cluster(cluster_addr(mine + 4 * x + k, (uint32_t)p));
        cluster_sync_all();  // nobody's shared memory goes while it is read
    }
    if (rank == 0 && y == 0) {
        float *w = a.weights + (int64_t)b * a.w_seq + (int64_t)hk * a.w_head + first + 4 * x, was[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) was[k] = first + 4 * x + k <= last ? w[k] : 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (first + 4 * x + k <= last) w[k] = was[k] + v[k];
    }
}

// Few columns (a decode step): keys go from memory to registers, a warp 32 / COLS of them at once, a
// lane W channels of each 32 W; queries wait in shared memory.  A lane's 32 sums (key, column) become
// one through five exchanges that halve them, lane l keeping key l / COLS and column l % COLS.
constexpr int kFewSpan = 64;  // a CTA takes a multiple of these keys

template <int W>
struct Channels {
    float v[W];
    __device__ __forceinline__ void load(const float *p, bool vec) {
        if constexpr (W == 4) {
            if (vec) {
                const float4 x = __ldg(reinterpret_cast<const float4 *>(p));
                v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
                return;
            }
        } else {
            if (vec) {
                const float2 x = __ldg(reinterpret_cast<const float2 *>(p));
                v[0] = x.x, v[1] = x.y;
                return;
            }
        }
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = __ldg(p + i);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = 0.f;
    }
};

template <int COLS, int W, bool CAP>
__global__ void __launch_bounds__(kF32Threads, 4) key_weights_few_kernel(const KeyWeightsArgs a, int span) {
    constexpr int kKeys = 32 / COLS, kWarps = kF32Threads / 32;
    extern __shared__ __align__(16) float sQ[];  // [COLS][chunks * 32 W], zeros where there is nothing
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.y / a.n_kv_heads, hk = blockIdx.y % a.n_kv_heads, G = a.n_heads / a.n_kv_heads, D = a.head_dim;
    const int raw = a.kv_lens[b], cols = a.n_q * G;
    if (raw < 0 || raw > a.max_kv_len) {
        if (blockIdx.x == 0 && hk == 0 && tid == 0) report_status(a.status, kErrBounds);
        return;
    }
    const int64_t off = (int64_t)raw - a.n_q, from = (int64_t)blockIdx.x * span;
    const int end = (int)min(from + span, (int64_t)raw);
    // the first key that some row sees
    const int first = (int)max(from, a.window > 0 ? off - a.window + 1 : (int64_t)0);
    if (first >= end) return;
    const int n = end - first;
    const int chunks = (D + 32 * W - 1) / (32 * W), pitch = chunks * 32 * W;
    const float *kb = static_cast<const float *>(a.k) + (int64_t)b * a.k_seq + (int64_t)hk * a.k_head;
    const float *qb = static_cast<const float *>(a.q) + (int64_t)b * a.n_q * a.q_rs + (int64_t)hk * G * D;

    // group g of this CTA's keys: first + g kKeys ...; this warp's are warp, warp + kWarps, ...
    Channels<W> held[kKeys];
    auto ask = [&](int g, int chunk) {
        const int d = (chunk * 32 + lane) * W;
#pragma unroll
        for (int k = 0; k < kKeys; ++k) {
            if (g * kKeys + k < n && d < D) held[k].load(kb + (int64_t)(first + g * kKeys + k) * a.k_row + d, a.k_vec);
            else held[k].zero();
        }
    };
    ask(warp, 0);
    for (int i = tid; i < COLS * pitch; i += kF32Threads) {
        const int c = i / pitch, d = i - c * pitch, row = c / G;
        sQ[i] = c < cols && d < D ? __ldg(qb + (int64_t)row * a.q_rs + (int64_t)(c - row * G) * D + d) : 0.f;
    }
    // this lane's column
    const int col = lane % COLS, my_row = col / G;
    float lse2 = INFINITY;
    int hi = -1, lo = -1;
    if (col < cols) {
        const float l = a.lse[((int64_t)b * a.n_q + my_row) * a.n_heads + hk * G + col - my_row * G];
        const int64_t pos = off + my_row;
        if (l != -INFINITY && pos >= 0) {
            lse2 = l * 1.4426950408889634f;
            hi = a.causal ? (int)pos : 0x7fffffff;
            lo = a.window > 0 ? (int)(pos - a.window) : -1;
        }
    }
    __syncthreads();
    float *w = a.weights + (int64_t)b * a.w_seq + (int64_t)hk * a.w_head;
    for (int g = warp; g * kKeys < n; g += kWarps) {
        float s[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) s[i] = 0.f;
        for (int chunk = 0; chunk < chunks; ++chunk) {
            Channels<W> k[kKeys];
#pragma unroll
            for (int i = 0; i < kKeys; ++i) k[i] = held[i];
            if (chunk + 1 < chunks) ask(g, chunk + 1);
            else ask(g + kWarps, 0);
#pragma unroll
            for (int c = 0; c < COLS; ++c) {
                Channels<W> q;
                const float *at = sQ + c * pitch + (chunk * 32 + lane) * W;
                if constexpr (W == 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(at);
                    q.v[0] = x.x, q.v[1] = x.y, q.v[2] = x.z, q.v[3] = x.w;
                } else {
                    const float2 x = *reinterpret_cast<const float2 *>(at);
                    q.v[0] = x.x, q.v[1] = x.y;
                }
#pragma unroll
                for (int i = 0; i < kKeys; ++i)
#pragma unroll
                    for (int e = 0; e < W; ++e) s[i * COLS + c] = fmaf(k[i].v[e], q.v[e], s[i * COLS + c]);
            }
        }
#pragma unroll
        for (int half = 16; half > 0; half >>= 1) {
            const bool upper = lane & half;
#pragma unroll
            for (int i = 0; i < half; ++i) {
                const float keep = upper ? s[i + half] : s[i], give = upper ? s[i] : s[i + half];
                s[i] = keep + __shfl_xor_sync(0xffffffffu, give, half);
            }
        }
        const int i = g * kKeys + lane / COLS, j = first + i;
        const float x = CAP ? a.cap_log2 * tanhf(s[0] * a.raw_over_cap) - lse2 : fmaf(s[0], a.scale_log2, -lse2);
        float p = i < n && j <= hi && j > lo ? fast_exp2(x) : 0.f;
#pragma unroll
        for (int o = 1; o < COLS; o <<= 1) p += __shfl_xor_sync(0xffffffffu, p, o);
        if (col == 0 && p != 0.f) atomicAdd(w + j, p);  // (this lane alone has the key; p is 0 where there is none)
    }
}

template <int D>
int held_cols() { return KwCfg<D>::kHeldCols; }

template <int D, bool CAP>
cudaError_t launch_tc(const KeyWeightsArgs &a, int grid, cudaStream_t s) {
    using C = KwCfg<D>;
    static SharedLimit limit;
    const cudaError_t e = limit(key_weights_kernel<D, CAP>, C::kSmem);
    if (e != cudaSuccess) return e;
    key_weights_kernel<D, CAP><<<grid, kThreads, C::kSmem, s>>>(a);
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
    } else if (G <= kMaxCols) {
        p->heads_per = G;
        p->rows_per = std::min(n_q, kMaxCols / G);
        p->head_blocks = 1;
    } else {
        p->heads_per = kMaxCols;
        p->rows_per = 1;
        p->head_blocks = (G + kMaxCols - 1) / kMaxCols;
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

cudaError_t launch_key_weights_f32(const KeyWeightsArgs &a, int num_sms, cudaStream_t s) {
    // (one block of nothing still sees the lengths)
    dim3 grid((unsigned)((std::max<int64_t>(a.max_kv_len, 1) + kF32Keys - 1) / kF32Keys), (unsigned)(a.batch * a.n_kv_heads));
    const bool cap = a.cap_log2 > 0.f;
    const int64_t cols = (int64_t)a.n_q * (a.n_heads / a.n_kv_heads);
    // no more columns at once than there are; CTAs share them while the SMs have room for four each
    auto go = [&](auto kernel, auto shared, int columns) {
        int log2 = 0;
        while (log2 < 3 && ((int64_t)grid.x * grid.y << (log2 + 1)) <= 4 * (int64_t)num_sms && ((int64_t)columns << log2) < cols) ++log2;
        if (log2 == 0) {
            kernel<<<grid, kF32Threads, 0, s>>>(a, 0);
            return cudaGetLastError();
        }
        grid.x <<= log2;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 1u << log2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.gridDim = grid;
        cfg.blockDim = dim3(kF32Threads);
        cfg.stream = s;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, shared, a, log2);
    };
    if (cols <= 8) {
        // longer stretches a CTA while there are eight CTAs an SM all the same (32 caches of 4096, head_dim
        // 128: 34 us; down to two CTAs an SM 42, sixteen 42)
        int span = kFewSpan;
        while (span < 1024 && ((int64_t)a.max_kv_len + 2 * span - 1) / (2 * span) * grid.y >= 8 * (int64_t)num_sms) span *= 2;
        const int width = a.head_dim == 64 ? 2 : 4, pitch = (a.head_dim + 32 * width - 1) / (32 * width) * 32 * width;
        auto few = [&](auto kernel, int columns) {
            kernel<<<dim3((unsigned)((std::max<int64_t>(a.max_kv_len, 1) + span - 1) / span), grid.y), kF32Threads,
                     columns * pitch * sizeof(float), s>>>(a, span);
        };
        if (cols <= 4 && width == 2) cap ? few(key_weights_few_kernel<4, 2, true>, 4) : few(key_weights_few_kernel<4, 2, false>, 4);
        else if (cols <= 4) cap ? few(key_weights_few_kernel<4, 4, true>, 4) : few(key_weights_few_kernel<4, 4, false>, 4);
        else if (width == 2) cap ? few(key_weights_few_kernel<8, 2, true>, 8) : few(key_weights_few_kernel<8, 2, false>, 8);
        else cap ? few(key_weights_few_kernel<8, 4, true>, 8) : few(key_weights_few_kernel<8, 4, false>, 8);
        return cudaGetLastError();
    }
    const cudaError_t e = cols <= 32 ? cap ? go(key_weights_f32_kernel<32, true, false>, key_weights_f32_kernel<32, true, true>, 32) : go(key_weights_f32_kernel<32, false, false>, key_weights_f32_kernel<32, false, true>, 32)
                          : cap      ? go(key_weights_f32_kernel<64, true, false>, key_weights_f32_kernel<64, true, true>, 64)
                                     : go(key_weights_f32_kernel<64, false, false>, key_weights_f32_kernel<64, false, true>, 64);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace lat
