// kv_q8.cu — rows into and out of an 8-bit KV cache (the record: q8_block.cuh).
//
// append: a team (a warp, four or sixteen, by what a block's new rows need) takes K or V of one
// (sequence, touched block, KV head).  It reads the block's new rows once into registers, reduces
// their largest magnitude, raises the stored scale's exponent where a block begun earlier needs it
// (then brings the codes before the new rows to the new scale), and writes the codes.  Rows that
// do not fit the registers are read again.
// expand: a thread takes one 16-byte part of a row, so that a warp reads and writes whole lines (four
// rows a thread 28.6 us, two 26.9, one 26.5 for 512 rows in and 2048 back, eight sequences).
// What bounds them: HBM on whole chunks (head_dim 128, blocks of 64: 64 % of the copy rate, of which
// the way back is two thirds); the launch on single tokens.
#include <algorithm>

#include "cache_kernels.h"
#include "device_common.cuh"
#include "q8_block.cuh"

namespace lat {

namespace {

// eight elements of a row
template <typename T>
struct Octet;
template <>
struct Octet<__nv_bfloat16> {
    uint4 w;
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, bool vec) {
        if (vec) {
            w = __ldg(reinterpret_cast<const uint4 *>(p));
        } else {
            const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
            w = make_uint4(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16, h[4] | (uint32_t)h[5] << 16,
                           h[6] | (uint32_t)h[7] << 16);
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(x[i] << 16), v[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
    }
};
template <>
struct Octet<float> {
    float4 x, y;
    __device__ __forceinline__ void zero() { x = y = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void load(const float *p, bool vec) {
        if (vec) {
            x = __ldg(reinterpret_cast<const float4 *>(p));
            y = __ldg(reinterpret_cast<const float4 *>(p) + 1);
        } else {
            x = make_float4(p[0], p[1], p[2], p[3]);
            y = make_float4(p[4], p[5], p[6], p[7]);
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
    }
};

constexpr int kThreads = 128;
template <typename T>
constexpr int kHeld = sizeof(T) == 2 ? 8 : 4;  // octets of a thread in registers: 32 words

// the codes of one part at another scale: `by` a power of two below one
__device__ __forceinline__ uint32_t rescaled(uint32_t w, float by) {
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t h = e4m3x2_to_f16x2((uint16_t)(w >> (16 * i)));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        out |= (uint32_t)to_e4m3x2(f.x * by, f.y * by) << (16 * i);
    }
    return out;
}

template <typename T, int D, int TEAM>
__global__ void __launch_bounds__(TEAM > kThreads ? TEAM : kThreads) append_q8_kernel(const Q8StoreArgs a) {
    constexpr int kOcts = D / 8, kTeams = TEAM > kThreads ? 1 : kThreads / TEAM, kRow = 2 * D;
    __shared__ float most[(TEAM > kThreads ? TEAM : kThreads) / 32];
    const int t = threadIdx.x % TEAM;
    const int64_t unit = (int64_t)blockIdx.x * kTeams + threadIdx.x / TEAM;
    if (TEAM == 32 && unit >= a.units) return;  // (a warp by itself; a CTA has one unit)
    const int which = (int)(unit & 1);
    uint32_t u = (uint32_t)(unit >> 1), bm, hk, b, m;
    bm = a.by_heads.div(u);
    hk = u - bm * a.n_kv_heads;
    b = a.by_touched.div(bm);
    m = bm - b * a.touched;
    const int pos = a.pos[b];
    if (pos < 0 || pos > a.capacity - a.n) {
        if (t == 0 && m == 0 && hk == 0) report_status(a.status, kErrBounds);
        return;
    }
    const int n = (pos >> a.block_shift) + (int)m;  // the block
    if (n > (pos + a.n - 1) >> a.block_shift) return;  // (not reached: there may be none, nor an int for its rows)
    const int first = n << a.block_shift;  // its first row
    const int lo = max(pos, first), hi = first + min(pos + a.n - first, 1 << a.block_shift);
    const T *src = static_cast<const T *>(which ? a.v : a.k) + ((int64_t)b * a.n + (lo - pos)) * a.rs + (int64_t)hk * D;
    unsigned char *rec = a.cache + (int64_t)b * a.cache_seq + (int64_t)n * a.cache_block + (int64_t)hk * a.cache_head;
    float *scale = reinterpret_cast<float *>(rec + ((int64_t)kRow << a.block_shift)) + which;
    const bool begun = lo > first;
    const int was = begun ? q8_exponent(*scale) : kQ8MinExp;

    // ---- the largest finite magnitude ---------------------------------------------------
    const int octs = (hi - lo) * kOcts;
    Octet<T> held[kHeld<T>];
#pragma unroll
    for (int i = 0; i < kHeld<T>; ++i) {
        const int x = t + i * TEAM;
        if (x < octs) held[i].load(src + (int64_t)(x / kOcts) * a.rs + x % kOcts * 8, a.vec);
        else held[i].zero();
    }
    float top = 0.f;
    auto raise = [&](const Octet<T> &o) {
        float v[8];
        o.get(v);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float x = fabsf(v[k]);
            top = fmaxf(top, x < INFINITY ? x : 0.f);
        }
    };
#pragma unroll
    for (int i = 0; i < kHeld<T>; ++i) raise(held[i]);
    for (int x = t + kHeld<T> * TEAM; x < octs; x += TEAM) {
        Octet<T> o;
        o.load(src + (int64_t)(x / kOcts) * a.rs + x % kOcts * 8, a.vec);
        raise(o);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if constexpr (TEAM > 32) {
        if ((t & 31) == 0) most[t >> 5] = top;
        __syncthreads();  // (everyone has read the old scale, too)
#pragma unroll
        for (int w = 0; w < TEAM / 32; ++w) top = fmaxf(top, most[w]);
    } else {
        __syncwarp();
    }
    const int e = max(was, q8_exponent_for(top));
    const float inv = two_to(-e);

    // ---- codes ----------------------------------------------------------------------------
    auto store = [&](const Octet<T> &o, int x) {
        float v[8];
        o.get(v);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = fmaf(v[k], 0.f, v[k] * inv);  // (an infinity becomes NaN)
        const int row = lo - first + x / kOcts;
        uint2 w;
        w.x = to_e4m3x2(v[0], v[1]) | (uint32_t)to_e4m3x2(v[2], v[3]) << 16;
        w.y = to_e4m3x2(v[4], v[5]) | (uint32_t)to_e4m3x2(v[6], v[7]) << 16;
        *reinterpret_cast<uint2 *>(rec + (int64_t)row * kRow + q8_place<D>(which * D + x % kOcts * 8, row)) = w;
    };
#pragma unroll
    for (int i = 0; i < kHeld<T>; ++i)
        if (t + i * TEAM < octs) store(held[i], t + i * TEAM);
    for (int x = t + kHeld<T> * TEAM; x < octs; x += TEAM) {
        Octet<T> o;
        o.load(src + (int64_t)(x / kOcts) * a.rs + x % kOcts * 8, a.vec);
        store(o, x);
    }
    if (begun && e > was) {  // the rows before
        const float by = two_to(max(-126, was - e));  // (2^-126 of any code is nothing)
        for (int x = t; x < (lo - first) * kOcts; x += TEAM) {
            const int row = x / kOcts;
            uint2 *p = reinterpret_cast<uint2 *>(rec + (int64_t)row * kRow + q8_place<D>(which * D + x % kOcts * 8, row));
            uint2 w = *p;
            w.x = rescaled(w.x, by), w.y = rescaled(w.y, by);
            *p = w;
        }
    }
    if (t == 0 && (!begun || e > was)) *scale = two_to(e);
}

// the sixteen values of a part, s times its codes, into T's memory
template <typename T>
__device__ __forceinline__ void put16(T *dst, const uint32_t (&w)[4], float s, bool vec) {
    float v[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t h = e4m3x2_to_f16x2((uint16_t)(w[i / 2] >> (16 * (i & 1))));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        v[2 * i] = f.x * s, v[2 * i + 1] = f.y * s;
    }
    if (!vec) {
#pragma unroll
        for (int i = 0; i < 16; ++i) dst[i] = T(v[i]);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            reinterpret_cast<float4 *>(dst)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            reinterpret_cast<uint4 *>(dst)[i] =
                make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                           pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
    }
}

constexpr int kExpandThreads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kExpandThreads) expand_q8_kernel(const Q8StoreArgs a) {
    constexpr int kParts = D / 8, kRows = kExpandThreads / kParts, kRow = 2 * D;  // rows of a CTA
    const int p = threadIdx.x % kParts, r = threadIdx.x / kParts, which = p >= kParts / 2;
    const int64_t x = (int64_t)blockIdx.x * kRows + r;  // a row of one head
    if (r >= kRows || x >= a.units) return;
    const uint32_t bt = a.by_heads.div((uint32_t)x), hk = (uint32_t)x - bt * a.n_kv_heads;
    const uint32_t b = a.by_n.div(bt), t = bt - b * a.n;
    const int pos = a.pos[b];
    if (pos < 0 || pos > a.capacity - a.n) {
        if (p == 0 && t == 0 && hk == 0) report_status(a.status, kErrBounds);
        return;
    }
    const int j = pos + (int)t, n = j >> a.block_shift, row = j & ((1 << a.block_shift) - 1);
    const unsigned char *rec = a.cache + (int64_t)b * a.cache_seq + (int64_t)n * a.cache_block + (int64_t)hk * a.cache_head;
    const uint4 w = __ldg(reinterpret_cast<const uint4 *>(rec + (int64_t)row * kRow + q8_place<D>(16 * p, row)));
    const float s = __ldg(reinterpret_cast<const float *>(rec + ((int64_t)kRow << a.block_shift)) + which);
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
    put16(static_cast<T *>(which ? a.v_out : a.k_out) + (int64_t)bt * a.rs + (int64_t)hk * D + 16 * (p - which * (kParts / 2)),
          words, s, a.vec != 0);
}

template <typename T, int D>
cudaError_t launch(const Q8StoreArgs &a, bool expand, cudaStream_t s) {
    if (expand) {
        constexpr int per = kExpandThreads / (D / 8);
        expand_q8_kernel<T, D><<<(unsigned)((a.units + per - 1) / per), kExpandThreads, 0, s>>>(a);
        return cudaGetLastError();
    }
    // A block's new rows fit a warp's registers, or those of a CTA, or are less than twice that and are
    // read again (cheaper than a CTA of 512: fp32, head_dim 128, blocks of 64 47.9 us, so 49.8), or take
    // 512 (head_dim 512: 28.2, read again 35.3).  A CTA on what a warp can hold: blocks of 16
    // 33.4 us, by warps 26.9.  (512 rows in, 2048 back, eight sequences of eight heads)
    const int64_t octs = (int64_t)std::min(a.n, 1 << a.block_shift) * (D / 8);
    if (octs <= 32 * kHeld<T>)
        append_q8_kernel<T, D, 32><<<(unsigned)((a.units + kThreads / 32 - 1) / (kThreads / 32)), kThreads, 0, s>>>(a);
    else if (octs <= 2 * kThreads * kHeld<T>)
        append_q8_kernel<T, D, kThreads><<<(unsigned)a.units, kThreads, 0, s>>>(a);
    else
        append_q8_kernel<T, D, 512><<<(unsigned)a.units, 512, 0, s>>>(a);
    return cudaGetLastError();
}
template <typename T>
cudaError_t launch_t(const Q8StoreArgs &a, bool expand, cudaStream_t s) {
    switch (a.head_dim) {
        case 64: return launch<T, 64>(a, expand, s);
        case 80: return launch<T, 80>(a, expand, s);
        case 128: return launch<T, 128>(a, expand, s);
        case 256: return launch<T, 256>(a, expand, s);
        case 512: return launch<T, 512>(a, expand, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_q8_store(const Q8StoreArgs &a, bool bf16, bool expand, cudaStream_t s) {
    return bf16 ? launch_t<__nv_bfloat16>(a, expand, s) : launch_t<float>(a, expand, s);
}

}  // namespace lat
