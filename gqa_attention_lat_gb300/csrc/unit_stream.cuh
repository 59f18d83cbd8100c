// unit_stream.cuh — the work of a split-KV decode over a packed cache as one stream of tiles.
//
// Work unit = one (sequence, KV head, block of <= 8 query heads).  All units' keys, laid end to
// end in tiles, form one stream; CTA c takes the c-th equal share (to a tile, never under
// min_tiles).  A unit cut across CTAs leaves one normalised partial and its log-sum-exp per
// piece.  The CTA that finishes a unit's last piece (an atomic ticket) joins them after its
// stream; units of many pieces are joined by a second kernel instead (split_join.cuh).
#pragma once

#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "cache_kernels.h"
#include "device_common.cuh"

namespace lat {

constexpr int kHeads = 8;                  // N of the mma: query heads of a unit
constexpr float kRescaleBy = 8.0f;         // log2 units the maximum may grow unnoticed
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kPieceRing = 8;              // pieces known ahead
// What a unit costs beside its tiles (its queries made ready, the warps' states joined), in
// tiles: counted in the shares, so that a CTA of many short units is not the last to finish (32
// sequences of 1 to 4096 keys, 4-bit cache: not counted 36.8 us, as 2 tiles 30.5 us).
constexpr int kUnitCost = 2;

struct Piece {
    int b, hk, hb;     // unit
    int key0, keys;    // first key, keys of the piece (the last tile may be partial)
    int slot, nseg;    // which piece of how many
    int end;           // no more pieces
};

struct Join {          // a unit cut across CTAs that this one may have to join
    int b, h_base, g_cnt, nseg, unit, last;
};

// The visible keys of a sequence, from the last multiple of Align at or before the first (the
// rows between are there and masked)
struct KeyRange {
    int lo, n;
};
template <int Align>
__device__ __forceinline__ KeyRange range_of(const SplitDecodeArgs &a, int len) {
    KeyRange k{0, 0};
    if (len < 0 || len > a.max_kv_len) return k;  // reported once, by CTA 0
    k.lo = a.window > 0 ? max(0, len - a.window) / Align * Align : 0;
    k.n = len - k.lo;
    return k;
}

// The stream of `total` tiles in equal shares: the first `more` CTAs have each + 1, the others each
struct Shares {
    uint32_t each, more;
    __device__ __forceinline__ uint32_t begin(uint32_t c) const { return each * c + min(c, more); }
    __device__ __forceinline__ uint32_t of(uint32_t x) const {  // whose tile x is
        const uint32_t b = more * (each + 1);
        return x < b ? x / (each + 1) : more + (x - b) / each;
    }
};
// thread 0's place in the stream
struct Walk {
    uint32_t pos, end, pb;  // pb: where sequence b's units begin
    Shares shares;
    int b;
};
struct StreamState {  // in shared memory
    Piece pieces[kPieceRing];
    Walk walk;
    uint32_t scan[4];  // a warp each
    int abort_flag;
    Join joins[2];
};

// a unit of n keys in the stream: nothing, or its tiles and what it costs beside them; where no
// unit is to be cut (a.whole), as much as the longest
template <int T>
__device__ __forceinline__ uint32_t tiles_of(int n) {
    return ((uint32_t)n + (T - 1)) / T;
}
template <int T>
__device__ __forceinline__ uint32_t unit_cost(const SplitDecodeArgs &a, int n) {
    return n <= 0 ? 0u : a.whole ? (uint32_t)a.min_tiles : tiles_of<T>(n) + kUnitCost;
}
template <int T, int Align>
__device__ bool next_piece(const SplitDecodeArgs &a, Walk &w, int HB, Piece &p) {
    const uint32_t HU = (uint32_t)(a.n_kv_heads * HB);
    while (w.pos < w.end && w.b < a.batch) {
        const KeyRange k = range_of<Align>(a, a.kv_lens[w.b]);
        const uint32_t cost = unit_cost<T>(a, k.n), nt = tiles_of<T>(k.n), all = cost * HU;
        if (w.pos >= w.pb + all) {
            w.pb += all;
            ++w.b;
            continue;
        }
        const uint32_t idx = (w.pos - w.pb) / cost, ustart = w.pb + idx * cost + kUnitCost;  // its first tile
        const uint32_t uend = ustart + nt;                                                       // behind its last
        const uint32_t t0 = w.pos > ustart ? w.pos - ustart : 0, t1 = w.end > ustart ? min(nt, w.end - ustart) : 0;
        const bool cut = w.pos > ustart;  // (divisions only for units that leave this share)
        w.pos = min(w.end, w.pb + (idx + 1) * cost);
        if (t0 >= t1) continue;  // the share ends before the unit's first tile
        const uint32_t first = cut ? w.shares.of(ustart) : blockIdx.x, last = uend > w.end ? w.shares.of(uend - 1) : blockIdx.x;
        p.b = w.b;
        p.hk = HB == 1 ? (int)idx : (int)(idx / HB);
        p.hb = HB == 1 ? 0 : (int)(idx % HB);
        p.key0 = k.lo + (int)t0 * T;
        p.keys = (int)(min((uint32_t)k.n, t1 * T) - t0 * T);
        p.slot = (int)(blockIdx.x - first);
        p.nseg = (int)(last - first + 1);
        p.end = 0;
        return true;
    }
    p.end = 1;
    return false;
}

// The stream's length in tiles of TK keys and this CTA's share: per-thread sums over a slice of
// the sequences, then a scan.  Sequences with nothing to stream get their zeros from CTA 0.  False
// for a CTA without a share; else the first piece stands in st.pieces[0].  Thread 0 calls `prepare`
// while lengths are under way, a barrier before anyone goes on.
template <int TK, int Align, int kWarps, typename T, typename Prepare>
__device__ __forceinline__ bool stream_begin(const SplitDecodeArgs &a, int HB, int D, StreamState &st, Prepare prepare) {
    constexpr int kThreads = 32 * kWarps;
    static_assert(kWarps <= 4, "st.scan");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, HU = a.n_kv_heads * HB;
    const int per_thread = (a.batch + kThreads - 1) / kThreads;
    const int b_lo = min(a.batch, tid * per_thread), b_hi = min(a.batch, b_lo + per_thread);
    uint32_t my_sum = 0;
    for (int b = b_lo; b < b_hi; ++b) {
        const int len = a.kv_lens[b];
        const KeyRange k = range_of<Align>(a, len);
        my_sum += unit_cost<TK>(a, k.n) * HU;
        if (blockIdx.x == 0 && k.n == 0) {  // nothing to stream
            const bool bad = len < 0 || len > a.max_kv_len;
            if (bad) report_status(a.status, kErrBounds);
            for (int h = 0; h < a.n_heads; ++h) {
                if (a.defer_join) a.piece_count[(int64_t)b * a.n_heads + h] = 0;
                if (!bad && a.lse != nullptr) a.lse[(int64_t)b * a.n_heads + h] = -INFINITY;
            }
            if (!bad)
                for (int i = 0; i < a.n_heads * D; ++i) static_cast<T *>(a.out)[(int64_t)b * a.out_rs + i] = T(0.f);
        }
    }
    uint32_t incl = my_sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
    }
    if (lane == 31) st.scan[warp] = incl;
    if (tid == 0) {
        st.walk.pos = 0;
        st.walk.end = 0;
        st.walk.b = a.batch;
        prepare();
        st.abort_flag = 0;
        st.joins[0].nseg = st.joins[1].nseg = st.joins[0].last = st.joins[1].last = 0;
    }
    __syncthreads();
    uint32_t total = 0, my_start = incl - my_sum;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const uint32_t v = st.scan[w];
        if (w < warp) my_start += v;
        total += v;
    }
    const uint32_t parts = max(1u, min(gridDim.x, total / (uint32_t)a.min_tiles)), each = total / parts;
    const Shares shares{each, total - each * parts};
    const uint32_t r0 = blockIdx.x < parts ? shares.begin(blockIdx.x) : 0;
    const uint32_t r1 = blockIdx.x < parts ? shares.begin(blockIdx.x + 1) : 0;
    if (r0 < r1 && r0 >= my_start && r0 - my_start < my_sum) {  // the share begins in this slice
        uint32_t p = my_start;
        int b = b_lo;
        for (; b < b_hi; ++b) {
            const uint32_t w = unit_cost<TK>(a, range_of<Align>(a, a.kv_lens[b]).n) * HU;
            if (r0 < p + w) break;
            p += w;
        }
        Walk w{r0, r1, p, shares, b};
        next_piece<TK, Align>(a, w, HB, st.pieces[0]);
        st.walk = w;
    }
    if (a.defer_join) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (r0 >= r1) return false;
    __syncthreads();
    return true;
}

__device__ __forceinline__ int add_acq_rel(int32_t *p, int x) {
    int was;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(was) : "l"(p), "r"(x) : "memory");
    return was;
}

// The units whose last piece was this CTA's: weights 2^{lse_c - lse} over their pieces.  After
// the stream, by all threads; nothing where a second kernel joins.
template <int D, bool F32, int kThreads>
__device__ __forceinline__ void stream_join(const SplitDecodeArgs &a, StreamState &st) {
    using T = typename std::conditional<F32, float, __nv_bfloat16>::type;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    volatile int *abort_flag = &st.abort_flag;
    if (a.defer_join) return;
    __syncthreads();  // every thread's partials are written
    if (*abort_flag) return;
    // (each thread's partials happen before the barrier, that before the ticket's release; a last
    // ticket's acquire before the next barrier, that before the reads, which skip L1)
    if (lane == 0 && warp < 2 && st.joins[warp].nseg > 0)  // a ticket a warp: they take a round trip each
        st.joins[warp].last = add_acq_rel(a.counters + st.joins[warp].unit, 1) == st.joins[warp].nseg - 1;
    __syncthreads();
    for (int k = 0; k < 2; ++k) {
        const Join j = st.joins[k];
        if (!j.last) continue;
        for (int v = tid; v < j.g_cnt * (D / 4); v += kThreads) {
            const int h = j.h_base + v / (D / 4), d = 4 * (v % (D / 4));
            const int64_t bh = (int64_t)j.b * a.n_heads + h;
            const float *pl = a.part_lse + bh * a.max_splits;
            const float *po = a.part_o + bh * a.max_splits * D + d;
            float m = -INFINITY, z = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            constexpr int kAhead = 8;  // pieces in flight
            for (int s0 = 0; s0 < j.nseg; s0 += kAhead) {
                float l[kAhead], mn = m;
                float4 w[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const bool there = s0 + i < j.nseg;
                    l[i] = there ? __ldcg(pl + s0 + i) : -INFINITY;
                    w[i] = there ? __ldcg(reinterpret_cast<const float4 *>(po + (int64_t)(s0 + i) * D))
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
                for (int i = 0; i < kAhead; ++i) mn = fmaxf(mn, l[i]);
                const float base = mn == -INFINITY ? 0.f : mn, cf = fast_exp2(m - base);
                z *= cf; o.x *= cf; o.y *= cf; o.z *= cf; o.w *= cf;
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const float e = fast_exp2(l[i] - base);
                    z += e;
                    o.x = fmaf(e, w[i].x, o.x); o.y = fmaf(e, w[i].y, o.y);
                    o.z = fmaf(e, w[i].z, o.z); o.w = fmaf(e, w[i].w, o.w);
                }
                m = mn;
            }
            const float rz = z == 0.f ? 0.f : 1.f / z;
            T *dst = static_cast<T *>(a.out) + (int64_t)j.b * a.out_rs + (int64_t)h * D + d;
            if constexpr (F32)
                *reinterpret_cast<float4 *>(dst) = make_float4(o.x * rz, o.y * rz, o.z * rz, o.w * rz);
            else
                *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(o.x * rz, o.y * rz), pack_bf16x2(o.z * rz, o.w * rz));
            if (d == 0 && a.lse != nullptr) a.lse[bh] = (m + log2f(z)) * kLn2;
        }
        if (tid == 0) a.counters[j.unit] = 0;  // ready for the next call
    }
}

__device__ __forceinline__ void mma_f16_16816(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// the power of two that brings m >= 0 to [2^to, 2^(to + 1)), as near as floats have one; 1 for
// nothing, NaN for what is not finite
__device__ __forceinline__ float to_f16_range(float m, int to) {
    const int e = (int)(__float_as_uint(m) >> 23);
    if (e == 255) return NAN;
    return m == 0.f ? 1.f : __uint_as_float((uint32_t)max(1, min(254, 127 + to + 127 - e)) << 23);
}

// of two magnitudes the larger, by their bits: a NaN is above all
__device__ __forceinline__ float larger_magnitude(float x, float y) {
    return __uint_as_float(max(__float_as_uint(x), __float_as_uint(y)));
}

// What `units` units of up to `range` tiles need on a grid of `grid` CTAs; false where a count
// passes 32 bits.  Fills everything of the plan but its grid.
inline bool plan_units(SplitPlan *p, int64_t units, int64_t range, int64_t rows, int head_dim) {
    // join grid: one CTA per (sequence, query head, up to 128 channels)
    if (rows * ((head_dim + 127) / 128) > 0x7fffffffLL) return false;
    // A unit of n tiles falls into at most n / min_tiles + 2 pieces.  min_tiles keeps that count
    // near 64 or, with few units, near the number of CTAs that each unit must feed.
    if (units * (range + kUnitCost) > 0x7fffffffLL) return false;
    const int64_t target = std::max<int64_t>(64, (p->grid + std::max<int64_t>(units, 1) - 1) / std::max<int64_t>(units, 1));
    p->min_tiles = (int)std::max<int64_t>(1, (range + target - 1) / target);
    // Units of up to two tiles, no more than the CTAs: one each, and nothing to join (4-bit cache,
    // 8 KV heads, head_dim 64: one sequence of 512 keys 7.3 instead of 8.0 us, 32 ragged ones of up
    // to 512 8.6 instead of 10.2; with three tiles it gains nothing).
    p->whole = range <= 2 && units <= p->grid;
    if (p->whole) p->min_tiles = (int)range + kUnitCost;
    p->max_splits = (int)((range + p->min_tiles - 1) / p->min_tiles) + 2;
    // With few units, cut finely, the CTA that joins one would read tens of partials after its
    // stream; a second kernel takes them then.
    p->defer_join = units * 8 < p->grid && p->max_splits > 16;
    auto round256 = [](size_t x) { return (x + 255) / 256 * 256; };
    p->part_o_bytes = round256((size_t)rows * p->max_splits * head_dim * 4);
    p->part_lse_bytes = round256((size_t)rows * p->max_splits * 4);
    // pieces per (sequence, head), or tickets per unit
    p->total_bytes = p->part_o_bytes + p->part_lse_bytes + round256((size_t)(p->defer_join ? rows : units) * 4);
    return true;
}

}  // namespace lat
