// block_select.cu — which blocks of a long cache a decode step reads.
//
// Bounds: for every block of block_size cached keys and every channel d, the largest and the
// smallest k_jd of the block, hi_d and lo_d (a row of 2 D numbers: the D maxima, the D minima).
// Score: no key of a block can score more against query head h than
//   u_h = sum_d max(q_hd hi_d, q_hd lo_d) = max(q, 0) . hi + min(q, 0) . lo,
// a product of length 2 D; a KV head's score of the block is the largest u_h of its heads.
// Choice: the n_first first blocks, the n_last last, and of the others the best scored, ties
// to the lowest, n_sel in all, in ascending order.
//
// The choice is that of the exact scores.  The score kernel works in fp32 and bounds its own
// error; the choosing kernel takes what lies further than that from the border as it is, and
// what lies nearer is scored again in pairs of floats (48 bits), so no rounding of a sum's order
// decides.
//
// What bounds them: bytes.  bounds reads each new key once, score each block's 2 D numbers
// once; the choice works on 4 bytes a block in shared memory and waits on barriers.
#include <math.h>

#include <algorithm>

#include "cache_kernels.h"
#include "device_common.cuh"

namespace lat {

namespace {

// -------------------------------------------------------------------------------- bounds
template <typename T>
struct Ext;
template <>
struct Ext<__nv_bfloat16> {  // eight channels: maxima and minima as packed pairs, NaN kept
    uint32_t hi[4], lo[4];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 4; ++i) hi[i] = 0xff80ff80u, lo[i] = 0x7f807f80u;  // -inf, +inf
    }
    static __device__ __forceinline__ uint32_t mx(uint32_t x, uint32_t y) {
        uint32_t r;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
        return r;
    }
    static __device__ __forceinline__ uint32_t mn(uint32_t x, uint32_t y) {
        uint32_t r;
        asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
        return r;
    }
};
template <>
struct Ext<float> {  // four channels
    uint32_t hi[4], lo[4];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 4; ++i) hi[i] = 0xff800000u, lo[i] = 0x7f800000u;
    }
    static __device__ __forceinline__ uint32_t mx(uint32_t x, uint32_t y) {
        float r;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(x)), "f"(__uint_as_float(y)));
        return __float_as_uint(r);
    }
    static __device__ __forceinline__ uint32_t mn(uint32_t x, uint32_t y) {
        float r;
        asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(x)), "f"(__uint_as_float(y)));
        return __float_as_uint(r);
    }
};

constexpr int kBoundWarps = 4;

// One warp per (sequence, touched block, KV head), heads fastest (their rows lie side by side in
// a token-major cache).  A row is kVecs 16-byte vectors: up to 32, a warp takes 32 / kVecs rows a
// load; beyond, a lane takes kPer vectors of a row.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kBoundWarps) block_bounds_kernel(const BoundsArgs a) {
    constexpr int kEl = 16 / (int)sizeof(T), kVecs = D / kEl;
    constexpr int kPer = kVecs > 32 ? kVecs / 32 : 1;
    constexpr int kLanes = kVecs / kPer;      // lanes of a row
    constexpr int kRows = 32 / kLanes;        // rows a load
    constexpr int kAhead = kPer >= 4 ? 2 : (kPer == 2 ? 4 : 8);  // loads in flight a lane and vector
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t u = blockIdx.x * kBoundWarps + warp;
    if (u >= (uint32_t)a.batch * a.max_touched * a.n_kv_heads) return;
    const uint32_t bt = u / a.n_kv_heads, hk = u - bt * a.n_kv_heads;
    const uint32_t b = bt / a.max_touched, t = bt - b * a.max_touched;
    const int p = a.pos[b];
    if (p < 0 || (int64_t)p + a.n_new > (int64_t)a.capacity) {
        if (t == 0 && hk == 0 && lane == 0) report_status(a.status, kErrBounds);
        return;
    }
    const int blk = p / a.block_size + (int)t;
    const int64_t first = (int64_t)blk * a.block_size;
    const int lo = (int)max((int64_t)p, first), hi = (int)min((int64_t)p + a.n_new, first + a.block_size);
    if (lo >= hi) return;
    const int row = lane / kLanes, col = lane % kLanes;
    const bool active = row < kRows;
    const unsigned char *k = static_cast<const unsigned char *>(a.k_cache) +
                             ((int64_t)b * a.cache_seq + (int64_t)hk * a.cache_head) * (int64_t)sizeof(T) + 16 * col;
    unsigned char *out = static_cast<unsigned char *>(a.bounds) +
                         ((int64_t)b * a.bounds_seq + (int64_t)blk * a.bounds_rs + (int64_t)hk * a.bounds_head) *
                             (int64_t)sizeof(T) + 16 * col;
    Ext<T> e[kPer];
#pragma unroll
    for (int v = 0; v < kPer; ++v) e[v].clear();
    if (lo > first && active && row == 0) {  // the block's earlier rows are in its stored bounds
#pragma unroll
        for (int v = 0; v < kPer; ++v) {
            const uint4 x = *reinterpret_cast<const uint4 *>(out + 16 * kLanes * v);
            const uint4 y = *reinterpret_cast<const uint4 *>(out + 16 * kLanes * v + D * sizeof(T));
            e[v].hi[0] = x.x, e[v].hi[1] = x.y, e[v].hi[2] = x.z, e[v].hi[3] = x.w;
            e[v].lo[0] = y.x, e[v].lo[1] = y.y, e[v].lo[2] = y.z, e[v].lo[3] = y.w;
        }
    }
    k += (int64_t)lo * a.cache_rs * (int64_t)sizeof(T);
    const int n = hi - lo;
    for (int j0 = 0; j0 < n; j0 += kRows * kAhead) {
        uint4 x[kAhead][kPer];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int j = min(j0 + i * kRows + row, n - 1);  // past the end: the last row again
#pragma unroll
            for (int v = 0; v < kPer; ++v)
                x[i][v] = active ? *reinterpret_cast<const uint4 *>(k + (int64_t)j * a.cache_rs * (int64_t)sizeof(T) + 16 * kLanes * v)
                                 : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int v = 0; v < kPer; ++v) {
                const uint32_t w[4] = {x[i][v].x, x[i][v].y, x[i][v].z, x[i][v].w};
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    e[v].hi[m] = Ext<T>::mx(e[v].hi[m], w[m]);
                    e[v].lo[m] = Ext<T>::mn(e[v].lo[m], w[m]);
                }
            }
    }
    // the row groups meet (kRows is 1, 2, 3 or 4): group 0 takes the others in turn
#pragma unroll
    for (int g = 1; g < kRows; ++g)
#pragma unroll
        for (int v = 0; v < kPer; ++v)
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const uint32_t h = __shfl_sync(0xffffffffu, e[v].hi[m], col + g * kLanes);
                const uint32_t l = __shfl_sync(0xffffffffu, e[v].lo[m], col + g * kLanes);
                e[v].hi[m] = row == 0 ? Ext<T>::mx(e[v].hi[m], h) : e[v].hi[m];
                e[v].lo[m] = row == 0 ? Ext<T>::mn(e[v].lo[m], l) : e[v].lo[m];
            }
    if (active && row == 0)
#pragma unroll
        for (int v = 0; v < kPer; ++v) {
            *reinterpret_cast<uint4 *>(out + 16 * kLanes * v) = make_uint4(e[v].hi[0], e[v].hi[1], e[v].hi[2], e[v].hi[3]);
            *reinterpret_cast<uint4 *>(out + 16 * kLanes * v + D * sizeof(T)) =
                make_uint4(e[v].lo[0], e[v].lo[1], e[v].lo[2], e[v].lo[3]);
        }
}

// --------------------------------------------------------------------------------- score
constexpr int kScoreWarps = 4;
constexpr int kScoreRows = 16;  // blocks a warp scores at a time
constexpr int kQHeads = 8;
// What the bounds of a score's error leave out: products and sums below the least normal number
// lose up to 2^-126 each, and there are 2 D of either at most
constexpr float kLeastError = 0x1p-115f;

__device__ __forceinline__ float max_nan(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

__device__ __forceinline__ int blocks_of(const SelectArgs &a, int b) {  // 0: nothing, or out of range
    const int len = a.kv_lens[b];
    return len <= 0 || len > a.max_kv_len ? 0 : (len - 1) / a.block_size + 1;
}

// CTA (unit, y): chunks y, y + gridDim.y, ... of 64 blocks of one (sequence, KV head).
// bf16: m16n8k16 with the blocks in M and up to 8 heads in N; lane (r, c) loads 16 bytes of
// rows r and r + 8 at column 8 (c + 4 i), which are the A fragments of two MMAs under a
// permutation of the columns that the queries share.  The same product over absolute values
// bounds the error: at most one unit in 2^-23 of that sum per addend.
template <int D>
__global__ void __launch_bounds__(32 * kScoreWarps) block_score_bf16_kernel(const SelectArgs a) {
    constexpr int kW = 2 * D, kSteps = kW / 32, kPitch = kW + 32;
    constexpr int kAhead = kSteps < 8 ? kSteps : 8;  // steps whose loads are in flight at once
    __shared__ __align__(16) __nv_bfloat16 sq[kQHeads][kPitch];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
    const int unit = blockIdx.x, b = unit / a.n_kv_heads, hk = unit % a.n_kv_heads;
    const int have = blocks_of(a, b), G = a.n_heads / a.n_kv_heads;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (have <= a.n_sel || (int64_t)blockIdx.y * kScoreWarps * kScoreRows >= have) return;  // all are kept, or not ours
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + (int64_t)b * a.q_rs + (int64_t)hk * G * D;
    const __nv_bfloat16 *bd = static_cast<const __nv_bfloat16 *>(a.bounds) + (int64_t)b * a.bounds_seq + (int64_t)hk * a.bounds_head;
    for (int h0 = 0; h0 < G; h0 += kQHeads) {
        bool staged = false;
        for (int chunk = blockIdx.y; chunk * kScoreWarps * kScoreRows < have; chunk += gridDim.y) {
            const int n0 = (chunk * kScoreWarps + warp) * kScoreRows;
            const uint4 *x = reinterpret_cast<const uint4 *>(bd + (int64_t)min(n0 + r, have - 1) * a.bounds_rs) + c;
            const uint4 *y = reinterpret_cast<const uint4 *>(bd + (int64_t)min(n0 + r + 8, have - 1) * a.bounds_rs) + c;
            uint4 vx[kAhead], vy[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) vx[i] = x[4 * i], vy[i] = y[4 * i];
            if (!staged) {  // the queries, while the first rows are on their way
                if (h0 > 0) __syncthreads();
                for (int i = tid; i < kQHeads * D / 8; i += 32 * kScoreWarps) {
                    const int h = i / (D / 8), d = 8 * (i % (D / 8));
                    const uint4 z = make_uint4(0, 0, 0, 0);
                    const uint4 w = h0 + h < G ? *reinterpret_cast<const uint4 *>(q + (h0 + h) * D + d) : z;
                    const uint32_t e[4] = {w.x, w.y, w.z, w.w};
                    uint32_t pos[4], neg[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {  // by the sign bit, channel by channel
                        const uint32_t m = ((e[k] >> 15) & 0x00010001u) * 0xffffu;
                        pos[k] = e[k] & ~m, neg[k] = e[k] & m;
                    }
                    *reinterpret_cast<uint4 *>(&sq[h][d]) = make_uint4(pos[0], pos[1], pos[2], pos[3]);
                    *reinterpret_cast<uint4 *>(&sq[h][D + d]) = make_uint4(neg[0], neg[1], neg[2], neg[3]);
                }
                __syncthreads();
                staged = true;
            }
            float s[4] = {0.f, 0.f, 0.f, 0.f}, t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i0 = 0; i0 < kSteps; i0 += kAhead) {
                if (i0 > 0)
#pragma unroll
                    for (int i = 0; i < kAhead; ++i)
                        if (i0 + i < kSteps) vx[i] = x[4 * (i0 + i)], vy[i] = y[4 * (i0 + i)];
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
                    if (i0 + i < kSteps) {
                        const uint4 w = *reinterpret_cast<const uint4 *>(&sq[r][32 * (i0 + i) + 8 * c]);
                        const uint32_t k = 0x7fff7fffu;
                        const uint32_t a0[4] = {vx[i].x, vy[i].x, vx[i].y, vy[i].y}, a1[4] = {vx[i].z, vy[i].z, vx[i].w, vy[i].w};
                        const uint32_t p0[4] = {a0[0] & k, a0[1] & k, a0[2] & k, a0[3] & k};
                        const uint32_t p1[4] = {a1[0] & k, a1[1] & k, a1[2] & k, a1[3] & k};
                        mma_bf16_16816(s, a0, w.x, w.y);
                        mma_bf16_16816(s, a1, w.z, w.w);
                        mma_bf16_16816(t, p0, w.x & k, w.y & k);
                        mma_bf16_16816(t, p1, w.z & k, w.w & k);
                    }
            }
            // the largest over the heads of this pass; a NaN wins
            const bool l0 = h0 + 2 * c < G, l1 = h0 + 2 * c + 1 < G;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float m = -INFINITY, e = 0.f;
                if (l0) m = s[2 * half], e = t[2 * half];
                if (l1) m = max_nan(m, s[2 * half + 1]), e = max_nan(e, t[2 * half + 1]);
#pragma unroll
                for (int off = 1; off < 4; off <<= 1) {
                    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
                    e = max_nan(e, __shfl_xor_sync(0xffffffffu, e, off));
                }
                const int n = n0 + r + 8 * half;
                if (c == 0 && n < have) {
                    float2 *dst = a.scores + (int64_t)unit * a.max_blocks + n;
                    e = fmaf(e, (2.f * D / 16.f + 1.f) * 18.f * 0x1p-23f, kLeastError);
                    if (h0 > 0) {  // more than eight heads: with what the earlier ones left
                        const float2 was = *dst;
                        m = max_nan(m, was.x), e = max_nan(e, was.y);
                    }
                    *dst = make_float2(m, e);
                }
            }
        }
    }
}

// fp32: a warp takes four blocks at a time, a lane 4 neighbouring columns of every 128; the 32
// sums of four blocks and eight heads come out of the lanes by a butterfly that halves the
// values at every step, one sum a lane.  The error bound: each addition is off by at most 2^-24
// of the sum of magnitudes, taken over the heads' largest |q|.
constexpr int kRowsF32 = 4;
template <int D>
__global__ void __launch_bounds__(32 * kScoreWarps) block_score_f32_kernel(const SelectArgs a) {
    constexpr int kW = 2 * D, kVecs = kW / 4, kSteps = (kVecs + 31) / 32;
    __shared__ __align__(16) float sq[kQHeads + 1][kW];  // the last: the largest |q| of the heads
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int unit = blockIdx.x, b = unit / a.n_kv_heads, hk = unit % a.n_kv_heads;
    const int have = blocks_of(a, b), G = a.n_heads / a.n_kv_heads;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (have <= a.n_sel || (int64_t)blockIdx.y * kScoreWarps * kRowsF32 >= have) return;
    const float *q = static_cast<const float *>(a.q) + (int64_t)b * a.q_rs + (int64_t)hk * G * D;
    const float *bd = static_cast<const float *>(a.bounds) + (int64_t)b * a.bounds_seq + (int64_t)hk * a.bounds_head;
    for (int h0 = 0; h0 < G; h0 += kQHeads) {
        if (h0 > 0) __syncthreads();
        for (int d = tid; d < D; d += 32 * kScoreWarps) {
            float hi = 0.f, lo = 0.f, x[kQHeads];
#pragma unroll
            for (int h = 0; h < kQHeads; ++h) x[h] = h0 + h < G ? q[(h0 + h) * D + d] : 0.f;
#pragma unroll
            for (int h = 0; h < kQHeads; ++h) {
                const bool neg = x[h] < 0.f;  // (a NaN goes with the maxima)
                sq[h][d] = neg ? 0.f : x[h];
                sq[h][D + d] = neg ? x[h] : 0.f;
                hi = fmaxf(hi, neg ? 0.f : x[h]);
                lo = fmaxf(lo, neg ? -x[h] : 0.f);
            }
            sq[kQHeads][d] = hi;
            sq[kQHeads][D + d] = lo;
        }
        __syncthreads();
        for (int chunk = blockIdx.y; chunk * kScoreWarps * kRowsF32 < have; chunk += gridDim.y) {
            const int n0 = (chunk * kScoreWarps + warp) * kRowsF32;
            float s[kRowsF32 * kQHeads], e[kRowsF32];
#pragma unroll
            for (int i = 0; i < kRowsF32 * kQHeads; ++i) s[i] = 0.f;
#pragma unroll
            for (int u = 0; u < kRowsF32; ++u) e[u] = 0.f;
#pragma unroll 2
            for (int v = 0; v < kSteps; ++v) {
                const int i = lane + 32 * v;
                if (i < kVecs) {
                    float4 w[kRowsF32];
#pragma unroll
                    for (int u = 0; u < kRowsF32; ++u)
                        w[u] = reinterpret_cast<const float4 *>(bd + (int64_t)min(n0 + u, have - 1) * a.bounds_rs)[i];
#pragma unroll
                    for (int h = 0; h <= kQHeads; ++h) {
                        const float4 y = *reinterpret_cast<const float4 *>(&sq[h][4 * i]);
#pragma unroll
                        for (int u = 0; u < kRowsF32; ++u) {
                            if (h < kQHeads) {
                                float &t = s[u * kQHeads + (h < kQHeads ? h : 0)];
                                t = fmaf(w[u].x, y.x, fmaf(w[u].y, y.y, fmaf(w[u].z, y.z, fmaf(w[u].w, y.w, t))));
                            } else {
                                e[u] = fmaf(fabsf(w[u].x), y.x, fmaf(fabsf(w[u].y), y.y, fmaf(fabsf(w[u].z), y.z, fmaf(fabsf(w[u].w), y.w, e[u]))));
                            }
                        }
                    }
                }
            }
            int off = 16;
#pragma unroll
            for (int half = kRowsF32 * kQHeads / 2; half >= 1; half /= 2, off /= 2) {
                const bool up = lane & off;
#pragma unroll
                for (int i = 0; i < half; ++i) {
                    const float keep = up ? s[i + half] : s[i], send = up ? s[i] : s[i + half];
                    s[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
                }
            }
            float err = 0.f;  // of this lane's block
#pragma unroll
            for (int u = 0; u < kRowsF32; ++u) {
#pragma unroll
                for (int k = 16; k > 0; k >>= 1) e[u] += __shfl_xor_sync(0xffffffffu, e[u], k);
                err = lane / kQHeads == u ? e[u] : err;
            }
            float m = h0 + lane % kQHeads < G ? s[0] : -INFINITY;
#pragma unroll
            for (int k = 1; k < kQHeads; k <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, k));
            const int n = n0 + lane / kQHeads;
            if (lane % kQHeads == 0 && n < have) {
                float2 *dst = a.scores + (int64_t)unit * a.max_blocks + n;
                err = fmaf(err, (kVecs / 8.f + 16.f) * 0x1p-23f, kLeastError);
                if (h0 > 0) {
                    const float2 was = *dst;
                    m = max_nan(m, was.x), err = max_nan(err, was.y);
                }
                *dst = make_float2(m, err);
            }
        }
    }
}

// -------------------------------------------------------------------------------- choose
constexpr int kPickWarps = 16;
constexpr int kPickThreads = 32 * kPickWarps;
constexpr int kPickWords = kSelectMaxBlocks / 32;

// scores as whole numbers in the same order; a NaN above all
__device__ __forceinline__ uint32_t order32(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);  // -0 as 0
    return x != x ? 0xffffffffu : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value32(uint32_t k) {
    return k == 0xffffffffu ? INFINITY : __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t order64(double x) {
    const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
    return x != x ? ~0ull : (u >> 63) ? ~u : u | (1ull << 63);
}

constexpr int kBins = kPickThreads;  // of one pass over the keys
constexpr int kFew = 512;            // candidates ranked in shared memory
constexpr int kBand = 8;             // of a bin that are scored exactly rather than binned again

struct PickShared {
    uint32_t in[kPickWords];   // chosen blocks, a bit each
    uint32_t tie[kPickWords];  // those near the border, then those equal to the last chosen one
    int red[kPickWarps];
    uint32_t red2[3][kPickWarps];
    int bins[kBins];
    int found, found_above, found_in;
    int few, sure;
    int at[kFew];
    uint64_t key[kFew];
};

__device__ __forceinline__ int block_sum(PickShared &sh, int x) {
    x = __reduce_add_sync(0xffffffffu, x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh.red[threadIdx.x >> 5] = x;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return __reduce_add_sync(0xffffffffu, lane < kPickWarps ? sh.red[lane] : 0);
}
// the least mn, and the largest mx and my
__device__ __forceinline__ void block_ends(PickShared &sh, uint32_t &mn, uint32_t &mx, uint32_t &my) {
    mn = __reduce_min_sync(0xffffffffu, mn);
    mx = __reduce_max_sync(0xffffffffu, mx);
    my = __reduce_max_sync(0xffffffffu, my);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
        const int w = threadIdx.x >> 5;
        sh.red2[0][w] = mn, sh.red2[1][w] = mx, sh.red2[2][w] = my;
    }
    __syncthreads();
    const int w = threadIdx.x % kPickWarps;
    mn = __reduce_min_sync(0xffffffffu, sh.red2[0][w]);
    mx = __reduce_max_sync(0xffffffffu, sh.red2[1][w]);
    my = __reduce_max_sync(0xffffffffu, sh.red2[2][w]);
}

// s + e = x + y exactly (Knuth's two-sum); the intrinsics keep the compiler from fusing
__device__ __forceinline__ float two_sum(float x, float y, float &e) {
    const float s = __fadd_rn(x, y), t = __fsub_rn(s, x);
    e = __fadd_rn(__fsub_rn(x, __fsub_rn(s, t)), __fsub_rn(y, t));
    return s;
}

// The block's score as a whole number in the scores' order, by a whole warp.  Products split by a
// fused multiply-add and sums by two-sum, each an unevaluated pair of floats: 48 bits on the fp32
// pipes.  A lane's 16 terms (at head_dim 512) and five joins leave 22 errors of 2^-24 of the terms'
// magnitudes in the lower float, whose 42 additions lose 2^-24 of it each: 2^-38 at most, nearer
// 2^-45 as they fall.  `fits` is cleared where the pair could overflow
// or lose small products; wide_score below is for those.  (fp64 runs at a 64th of fp32's rate
// here: scores in fp64 cost 13 us a step, only the pairs' last sums and comparisons in it 4.)
template <typename T>
__device__ uint64_t pair_score(const SelectArgs &a, int b, int hk, int n, bool &fits) {
    const int G = a.n_heads / a.n_kv_heads, D = a.head_dim, lane = threadIdx.x & 31;
    const T *q = static_cast<const T *>(a.q) + (int64_t)b * a.q_rs + (int64_t)hk * G * D;
    const T *x = static_cast<const T *>(a.bounds) + (int64_t)b * a.bounds_seq + (int64_t)hk * a.bounds_head + (int64_t)n * a.bounds_rs;
    uint64_t best = 0;
    for (int h0 = 0; h0 < G; h0 += 4) {
        float s[4] = {0.f, 0.f, 0.f, 0.f}, c[4] = {0.f, 0.f, 0.f, 0.f};
        float top = 0.f, other = 0.f;
#pragma unroll 2
        for (int d = lane; d < D; d += 32) {
            const float hi = (float)x[d], lo = (float)x[D + d];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float w = h0 + i < G ? (float)q[(h0 + i) * D + d] : 0.f, k = w < 0.f ? lo : hi;
                const float p = __fmul_rn(w, k);
                other = fmaf(w, w < 0.f ? hi : lo, other);
                float e;
                s[i] = two_sum(s[i], p, e);
                c[i] = __fadd_rn(c[i], __fadd_rn(e, __fmaf_rn(w, k, -p)));
                top = max_nan(top, fabsf(p));
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float e;
                const float c2 = __shfl_xor_sync(0xffffffffu, c[i], off);
                s[i] = two_sum(s[i], __shfl_xor_sync(0xffffffffu, s[i], off), e);
                c[i] = __fadd_rn(c[i], __fadd_rn(c2, e));
            }
            top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, off));
        }
        // (the products not taken count where they are no numbers: 0 times an infinite bound)
        if (!(top > 0x1p-60f && top < 0x1p100f) || other != other) fits = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // the nearest float and the rest: the pairs' order is the sums'
            float l;
            const float h = two_sum(s[i], c[i], l);
            const uint64_t key = (uint64_t)order32(h) << 32 | order32(l);
            if (h0 + i < G && key > best) best = key;
        }
    }
    return best;
}
template <typename T>
__device__ __noinline__ uint64_t wide_score(const SelectArgs &a, int b, int hk, int n) {
    const int G = a.n_heads / a.n_kv_heads, D = a.head_dim, lane = threadIdx.x & 31;
    const T *q = static_cast<const T *>(a.q) + (int64_t)b * a.q_rs + (int64_t)hk * G * D;
    const T *x = static_cast<const T *>(a.bounds) + (int64_t)b * a.bounds_seq + (int64_t)hk * a.bounds_head + (int64_t)n * a.bounds_rs;
    uint64_t best = 0;
    for (int h = 0; h < G; ++h) {
        double v = 0.0;
        for (int d = lane; d < D; d += 32) {
            const double w = (double)(float)q[h * D + d], hi = w * (double)(float)x[d], lo = w * (double)(float)x[D + d];
            const double other = w < 0.0 ? hi : lo;
            v += other != other ? other : w < 0.0 ? lo : hi;  // (exact products: no fma needed)
        }
        for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        const uint64_t key = order64(v);
        best = key > best ? key : best;
    }
    return best;
}

// One CTA per (sequence, KV head).  The k-th largest score is found by counting the ordered keys
// into 512 equal bins of the range that still holds it (the scores of one query lie within a few
// binades, so they spread over the bins).  It ends as soon as exactly k keys lie from some bin on,
// or few share the bin: those are scored exactly, as a near border needs anyway.  Measured on 64
// of up to 2048 blocks, 64 KV heads, score pass included: bins down to one key and sums ended in
// fp64 19.7 us, in float pairs 19.0, the few of a bin scored 17.7, the warps' results joined by
// one reduction instead of a loop 17.2.  What is left is barriers and first passes through code.
template <typename T>
__global__ void __launch_bounds__(kPickThreads) block_pick_kernel(const SelectArgs a) {
    extern __shared__ uint32_t keys[];  // [have - n_first - n_last] where they fit, else unused
    __shared__ PickShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int unit = blockIdx.x, b = unit / a.n_kv_heads, hk = unit % a.n_kv_heads;
    const int len = a.kv_lens[b];
    int32_t *out = a.blocks + (int64_t)unit * a.n_sel;
    if (len < 0 || len > a.max_kv_len) {  // left as it was
        if (tid == 0 && hk == 0) report_status(a.status, kErrBounds);
        return;
    }
    const int have = blocks_of(a, b);
    if (have <= a.n_sel) {  // all of them
        // (whole numbers without a sign: n_sel may be the largest int)
        for (uint32_t i = tid; i < (uint32_t)a.n_sel; i += kPickThreads) out[i] = i < (uint32_t)have ? (int)i : -1;
        return;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the scores are complete
    const float2 *scores = a.scores + (int64_t)unit * a.max_blocks;
    const int c0 = a.n_first, c1 = have - a.n_last, n = c1 - c0;  // the free choice
    const int k = a.n_sel - a.n_first - a.n_last;                 // how many of it; n > k
    const bool held = n <= a.keys_held;
    if (tid == 0) sh.few = sh.sure = 0;
    float e_max = 0.f;
    uint32_t top = 0, low = 0xffffffffu;
    for (int i = tid; i < n; i += kPickThreads) {
        const float2 s = __ldcg(scores + c0 + i);
        const uint32_t key = order32(s.x);
        if (held) keys[i] = key;
        low = min(low, key);
        top = max(top, key);
        e_max = s.y <= 3e38f ? fmaxf(e_max, s.y) : INFINITY;
    }
    uint32_t eu = __float_as_uint(e_max), unused = 0;
    block_ends(sh, low, top, eu);
    e_max = __uint_as_float(eu);
    auto key_at = [&](int i) { return held ? keys[i] : order32(__ldcg(scores + c0 + i).x); };
    // kth: the k-th largest key; next: the (k + 1)-th.  Where they share a bin with few others
    // (band): the bin's first and last key, which hold the k-th largest between them
    uint32_t kth = 0, next = 0;
    bool band = false;
    if (k > 0) {
        uint32_t lo = low;   // count(>= lo) is at_lo >= k; the k-th largest lies in the `width` keys from lo on
        int at_lo = n, above_all = 0;  // keys above that range
        uint32_t last = top - low;     // its width less one
        while (at_lo != k && last > 0) {
            const int shift = max(0, 32 - __clz(last) - 9);  // last >> shift < 512
            sh.bins[tid] = 0;
            __syncthreads();
            for (int i = tid; i < n; i += kPickThreads) {
                const uint32_t d = key_at(i) - lo;
                if (d <= last) atomicAdd(&sh.bins[d >> shift], 1);
            }
            __syncthreads();
            const int mine = sh.bins[tid];
            int from = mine;  // keys of this and the higher bins of the warp
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int v = __shfl_down_sync(0xffffffffu, from, off);
                if (lane + off < 32) from += v;
            }
            if (lane == 0) sh.red[warp] = from;
            __syncthreads();
            from += above_all + __reduce_add_sync(0xffffffffu, lane > warp && lane < kPickWarps ? sh.red[lane] : 0);
            if (from >= k && from - mine < k) sh.found = tid, sh.found_above = from - mine, sh.found_in = from;
            __syncthreads();
            lo += (uint32_t)sh.found << shift;
            above_all = sh.found_above;
            at_lo = sh.found_in;
            last = min(last - ((uint32_t)sh.found << shift), (1u << shift) - 1u);
            if (at_lo != k && at_lo - above_all <= kBand) {
                kth = lo, next = lo + last, band = true;
                break;
            }
        }
        if (!band) {
            uint32_t above = 0xffffffffu, below = 0;
            for (int i = tid; i < n; i += kPickThreads) {
                const uint32_t key = key_at(i);
                if (key >= lo) above = min(above, key);
                else below = max(below, key);
            }
            block_ends(sh, above, below, unused);
            kth = above;
            next = at_lo == k ? below : kth;  // more than k from lo on: they are equal to it
        }
    }
    // sure of its place: further than both errors from the other side of the border
    const float f_kth = value32(kth), f_next = value32(next);
    const float in_above = f_next + 2.f * e_max, out_below = f_kth - 2.f * e_max;
    const bool clear = k == 0 || (!band && next < kth && in_above < f_kth);
    int sures = 0;  // (of the warp)
    for (int w0 = warp; w0 * 32 < have; w0 += kPickWarps) {  // one word of 32 blocks
        const int i = w0 * 32 + lane, j = i - c0;
        bool in = i < have && (j < 0 || i >= c1), sure = false, maybe = false;
        if (!in && i < have && k > 0) {
            const uint32_t key = key_at(j);
            if (clear) {
                in = key >= kth;
            } else {
                const float f = value32(key);
                const bool nan = key == 0xffffffffu;
                in = sure = !nan && f > in_above && key > next;
                maybe = !in && (nan || !(f < out_below));
            }
        }
        const uint32_t bits = __ballot_sync(0xffffffffu, in);
        if (lane == 0) sh.in[w0] = bits;
        if (!clear) {
            sures += __popc(__ballot_sync(0xffffffffu, sure));
            const uint32_t may = __ballot_sync(0xffffffffu, maybe);
            if (lane == 0) sh.tie[w0] = may;
            if (maybe) {  // the first of them also as a list
                const int at = atomicAdd(&sh.few, 1);
                if (at < kFew) sh.at[at] = i;
            }
        }
    }
    if (lane == 0 && sures > 0) atomicAdd(&sh.sure, sures);
    __syncthreads();
    const int words = (have + 31) / 32;
    if (!clear) {
        const int need = k - sh.sure, cand = sh.few;
        if (need >= cand) {  // all of them (need is cand: no more than k are above the border)
            for (int w = tid; w < words; w += kPickThreads) sh.in[w] |= sh.tie[w], sh.tie[w] = 0;
        } else {
            // exact scores of the candidates.  A few (the usual case): each counts those ahead of it
            if (cand <= kFew) {
                bool fits = true;
                for (int i = warp; i < cand; i += kPickWarps) {
                    const uint64_t s = pair_score<T>(a, b, hk, sh.at[i], fits);
                    if (lane == 0) sh.key[i] = s;
                }
                if (__syncthreads_or(!fits)) {
                    for (int i = warp; i < cand; i += kPickWarps) {
                        const uint64_t s = wide_score<T>(a, b, hk, sh.at[i]);
                        if (lane == 0) sh.key[i] = s;
                    }
                    __syncthreads();
                }
                if (tid < cand) {
                    const uint64_t mine = sh.key[tid];
                    const int at = sh.at[tid];
                    int ahead = 0;
                    for (int i = 0; i < cand; ++i) ahead += sh.key[i] > mine || (sh.key[i] == mine && sh.at[i] < at);
                    if (ahead < need) atomicOr(&sh.in[at / 32], 1u << (at % 32));
                }
            } else {
                // many: the border among their ordered keys by halving, kept beside the scores
                uint64_t *exact = a.exact + (int64_t)unit * a.max_blocks;
                bool fits = true;
                for (int w = warp; w < words; w += kPickWarps)
                    for (uint32_t m = sh.tie[w]; m != 0; m &= m - 1) {
                        const int i = w * 32 + __ffs(m) - 1;
                        const uint64_t s = pair_score<T>(a, b, hk, i, fits);
                        if (lane == 0) exact[i] = s;
                    }
                if (__syncthreads_or(!fits)) {
                    for (int w = warp; w < words; w += kPickWarps)
                        for (uint32_t m = sh.tie[w]; m != 0; m &= m - 1) {
                            const int i = w * 32 + __ffs(m) - 1;
                            const uint64_t s = wide_score<T>(a, b, hk, i);
                            if (lane == 0) exact[i] = s;
                        }
                    __syncthreads();
                }
                uint64_t lo = 0, hi = ~0ull;  // the need-th largest lies in [lo, hi]
                int at_lo = cand;
                while (lo < hi && at_lo != need) {
                    const uint64_t mid = lo + (hi - lo) / 2 + 1;
                    int cnt = 0;
                    for (int w = tid; w < words; w += kPickThreads)
                        for (uint32_t m = sh.tie[w]; m != 0; m &= m - 1) cnt += exact[w * 32 + __ffs(m) - 1] >= mid;
                    cnt = block_sum(sh, cnt);
                    if (cnt >= need) lo = mid, at_lo = cnt;
                    else hi = mid - 1;
                }
                // above lo: in.  At lo: all when they are exactly as many, else the lowest first.
                int over = 0;
                for (int w = tid; w < words; w += kPickThreads) {
                    uint32_t in = 0, eq = 0;
                    for (uint32_t m = sh.tie[w]; m != 0; m &= m - 1) {
                        const int bit = __ffs(m) - 1;
                        const uint64_t x = exact[w * 32 + bit];
                        if (x > lo || (x == lo && at_lo == need)) in |= 1u << bit;
                        else if (x == lo) eq |= 1u << bit;
                        over += x > lo || (x == lo && at_lo == need);
                    }
                    sh.in[w] |= in;
                    sh.tie[w] = eq;
                }
                const int left = need - block_sum(sh, over);
                if (left > 0 && at_lo != need && warp == 0) {
                    int got = 0;
                    for (int w0 = 0; w0 < words && got < left; w0 += 32) {
                        const uint32_t eq = w0 + lane < words ? sh.tie[w0 + lane] : 0u;
                        int before = __popc(eq);
    #pragma unroll
                        for (int off = 1; off < 32; off <<= 1) {
                            const int v = __shfl_up_sync(0xffffffffu, before, off);
                            if (lane >= off) before += v;
                        }
                        const int all = __shfl_sync(0xffffffffu, before, 31);
                        int room = max(0, min(__popc(eq), left - got - (before - __popc(eq))));
                        uint32_t m = eq, take = 0;
                        for (; room > 0; --room, m &= m - 1) take |= m & (0u - m);
                        if (w0 + lane < words) sh.in[w0 + lane] |= take;
                        got += all;
                    }
                }
            }
        }
        __syncthreads();
    }
    // the chosen in ascending order
    for (int w0 = 0, base = 0; w0 < words; w0 += 32) {  // every warp counts, warp by warp writes
        const uint32_t in = w0 + lane < words ? sh.in[w0 + lane] : 0u;
        int before = __popc(in);
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, before, off);
            if (lane >= off) before += v;
        }
        const int all = __shfl_sync(0xffffffffu, before, 31);
        if ((w0 / 32) % kPickWarps == warp) {
            int at = base + before - __popc(in);
            for (uint32_t m = in; m != 0; m &= m - 1, ++at)
                if (at < a.n_sel) out[at] = (w0 + lane) * 32 + __ffs(m) - 1;
        }
        base += all;
    }
}

template <typename T>
cudaError_t launch_bounds_t(const BoundsArgs &a, unsigned blocks, cudaStream_t s) {
    constexpr int kT = 32 * kBoundWarps;
    switch (a.head_dim) {
        case 64: block_bounds_kernel<T, 64><<<blocks, kT, 0, s>>>(a); break;
        case 80: block_bounds_kernel<T, 80><<<blocks, kT, 0, s>>>(a); break;
        case 128: block_bounds_kernel<T, 128><<<blocks, kT, 0, s>>>(a); break;
        case 256: block_bounds_kernel<T, 256><<<blocks, kT, 0, s>>>(a); break;
        case 512: block_bounds_kernel<T, 512><<<blocks, kT, 0, s>>>(a); break;
        default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_score(const SelectArgs &a, bool bf16, dim3 grid, cudaStream_t s) {
    if (bf16)
        block_score_bf16_kernel<D><<<grid, 32 * kScoreWarps, 0, s>>>(a);
    else
        block_score_f32_kernel<D><<<grid, 32 * kScoreWarps, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_bounds(const BoundsArgs &a, bool bf16, cudaStream_t s) {
    const int64_t units = (int64_t)a.batch * a.max_touched * a.n_kv_heads;  // below 2^31
    const unsigned blocks = (unsigned)((units + kBoundWarps - 1) / kBoundWarps);
    return bf16 ? launch_bounds_t<__nv_bfloat16>(a, blocks, s) : launch_bounds_t<float>(a, blocks, s);
}

cudaError_t launch_select_blocks(SelectArgs a, bool bf16, int num_sms, cudaStream_t s) {
    const int units = a.batch * a.n_kv_heads;
    if (a.max_blocks > a.n_sel) {
        const int per = kScoreWarps * (bf16 ? kScoreRows : kRowsF32), chunks = (a.max_blocks + per - 1) / per;
        // enough CTAs for every SM to hold its fill; a CTA goes on with further chunks
        const int want = std::max(1, (16 * num_sms + units - 1) / units);
        const dim3 grid(units, std::min(chunks, want));
        cudaError_t e;
        switch (a.head_dim) {
            case 64: e = launch_score<64>(a, bf16, grid, s); break;
            case 80: e = launch_score<80>(a, bf16, grid, s); break;
            case 128: e = launch_score<128>(a, bf16, grid, s); break;
            case 256: e = launch_score<256>(a, bf16, grid, s); break;
            case 512: e = launch_score<512>(a, bf16, grid, s); break;
            default: return cudaErrorInvalidValue;
        }
        if (e != cudaSuccess) return e;
    }
    // the keys stay in shared memory up to 16 KB of them (beside 16 KB of bits), which
    // needs no attribute; beyond, every step reads them again from L2 (64 lists: of 2048 blocks
    // 22.1 us held and 24.1 read again, of 4096 34.2 and 39.0)
    a.keys_held = std::min(a.max_blocks, 4096);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = a.max_blocks > a.n_sel;
    cfg.gridDim = dim3((unsigned)units);
    cfg.blockDim = dim3(kPickThreads);
    cfg.dynamicSmemBytes = 4 * (size_t)a.keys_held;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = bf16 ? cudaLaunchKernelEx(&cfg, block_pick_kernel<__nv_bfloat16>, a)
                               : cudaLaunchKernelEx(&cfg, block_pick_kernel<float>, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace lat
