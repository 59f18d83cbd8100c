// kv_q4.cu — rows into and out of the 4-bit KV cache (the row format: q4_row.cuh).
//
// Append: rows pos[b] + t of sequence b's cache take the quantised new rows (t < n_new).
// Expand: rows pos[b] + t read back as K and V rows.  Both move bytes: 4 bytes a channel of
// bf16 K and V on one side, 1.25 on the other.
//
// How: a warp takes kRows head rows at once, so that their loads are in flight together, first
// all their K, then all their V.  A lane works on 8 neighbouring channels (an octet: one 16-byte
// vector of bf16), four lanes on a group.  K's octet is one word of the row.  V's octet is one
// nibble of eight halves: the four lanes of a group OR their nibbles together, or hand each
// other their halves.  Packed rows pass through shared memory, so that the cache is read and
// written in 16-byte vectors.  Both are bound by instruction issue as much as by bytes, so:
// codes leave a float through its own bits (an added 1.5 * 2^23 puts a whole number there),
// eight of them gather by a multiply-add each, and a head row's place comes by multiplication.
#include <math.h>

#include "cache_kernels.h"
#include "device_common.cuh"
#include "q4_row.cuh"

namespace lat {

namespace {

constexpr int kStoreWarps = 4;

__device__ __forceinline__ float min_nan(float x, float y) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float max_nan(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

// an octet of new channels as it lies in memory, so that many can be in flight
template <typename T>
struct Octet;
template <>
struct Octet<float> {
    float x[8];
    __device__ __forceinline__ void load(const float *p, bool vec) {
        if (vec) {
            const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
            x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = p[k];
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = 0.f;
    }
    __device__ __forceinline__ void get(float (&y)[8]) const {
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = x[k];
    }
    // the smallest and largest with zero among them; a NaN makes both NaN
    __device__ __forceinline__ void ends(float &mn, float &mx) const {
        mn = mx = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            mn = min_nan(mn, x[k]);
            mx = max_nan(mx, x[k]);
        }
    }
};
template <>
struct Octet<__nv_bfloat16> {
    uint32_t w[4];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, bool vec) {
        if (vec) {
            const uint4 a = *reinterpret_cast<const uint4 *>(p);
            w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[k] = (uint32_t)reinterpret_cast<const uint16_t *>(p)[2 * k] |
                       ((uint32_t)reinterpret_cast<const uint16_t *>(p)[2 * k + 1] << 16);
        }
    }
    __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0u; }
    __device__ __forceinline__ void get(float (&y)[8]) const {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            y[2 * k] = __uint_as_float(w[k] << 16);
            y[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void ends(float &mn, float &mx) const {
        uint32_t lo = 0u, hi = 0u;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(lo) : "r"(w[k]));
            asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(hi) : "r"(w[k]));
        }
        mn = min_nan(__uint_as_float(lo << 16), __uint_as_float(lo & 0xffff0000u));
        mx = max_nan(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u));
    }
};

// eight channels as bf16 pairs v of whole numbers times the scale s, rounded once
__device__ __forceinline__ void save8(__nv_bfloat16 *p, bool vec, const uint32_t v[4], uint32_t s2) {
    uint32_t y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 t = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&v[k]),
                                         *reinterpret_cast<const __nv_bfloat162 *>(&s2));
        y[k] = *reinterpret_cast<const uint32_t *>(&t);
    }
    if (vec) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(y[0], y[1], y[2], y[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            reinterpret_cast<uint16_t *>(p)[k] = (uint16_t)(y[k / 2] >> (16 * (k & 1)));
    }
}
__device__ __forceinline__ void save8(float *p, bool vec, const uint32_t v[4], uint32_t s2) {
    const float s = __uint_as_float(s2 & 0xffff0000u);
    float y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = s * __uint_as_float((k & 1) ? v[k / 2] & 0xffff0000u : v[k / 2] << 16);
    if (vec) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(y[0], y[1], y[2], y[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(y[4], y[5], y[6], y[7]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) p[k] = y[k];
    }
}

constexpr float kWhole = 12582912.f;  // 1.5 * 2^23: the sum's low bits are the whole number
constexpr uint32_t kWholeBits = 0x4b400000u;

// Codes of N channels, channel k at nibble k: c = nearest(x / s) + z in 0 .. 15, where the
// nearest whole number is that of the exact quotient, ties to even.  n = rint(x r) with r the
// rounded 1 / s is within one of it, and the remainder x - n s is exact in fp32 (s has 8 bits;
// for n = 0 it is x, and for n != 0 it ends no lower than x's last place and stays below 2 s).
template <int N>
__device__ __forceinline__ uint32_t codes_of(const float (&x)[N], float s, float r, float z) {
    static_assert(N == 1 || N == 8, "the constants' sum");
    const float half = 0.5f * s, z15 = z * (1.f / 15.f);
    float t[N], n[N], e[N];  // the whole number behind kWhole's bits, itself, the remainder
    bool near = false;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        t[k] = fmaf(x[k], r, kWhole);
        n[k] = t[k] - kWhole;
        e[k] = fmaf(-n[k], s, x[k]);
        near |= !(fabsf(e[k]) < half);
    }
    if (near) {  // some quotient at a half (the even one it is), or rounded the wrong way
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const bool odd = (__float_as_uint(t[k]) & 1u) != 0;
            if (fabsf(e[k]) > half || (fabsf(e[k]) == half && odd)) n[k] += copysignf(1.f, e[k]);
        }
    }
    uint32_t code = 0;
#pragma unroll
    for (int k = N - 1; k >= 0; --k)
        // held in 0 .. 15 as a fraction of 15 in 0 .. 1, whose rounding error times 15 is no half
        code = code * 16u + __float_as_uint(fmaf(__saturatef(fmaf(n[k], 1.f / 15.f, z15)), 15.f, kWhole));
    // each of them brought kWholeBits with it, times 16^k
    return code - kWholeBits * (N == 8 ? 0x11111111u : 1u);
}

// the nibbles of even number, then those of odd number
__device__ __forceinline__ uint32_t evens_first(uint32_t x) {
    const uint32_t t = (x ^ (x >> 4)) & 0x00f000f0u;  // nibbles 1 and 2 of each half change places
    return __byte_perm(x ^ t ^ (t << 4), 0, 0x3120);
}

template <int D>
struct StoreCfg {
    using R = Q4Row<D>;
    static constexpr int kRows = D == 80 ? 8 : D <= 128 ? 4 : D == 256 ? 2 : 1;  // a warp's head rows
    static constexpr int kOcts = R::kPad / 8;             // octets of a row's K (or V)
    static constexpr int kSteps = kRows * kOcts / 32;     // a lane's octets of K (or V)
    static_assert(kRows * kOcts % 32 == 0, "every lane has an octet in every step");
    static constexpr int kPieces = R::kBytes / 16;
};

// A warp's head rows: lane i < kRows finds row i's place, every lane asks for the row it works
// on.  `cache`: byte offset in the cache; `rows`: element offset among the new (or output) rows;
// -1 past the end, and in the cache where the sequence does not fit (reported once).
struct Places {
    int64_t cache, rows;
    __device__ __forceinline__ Places(const Q4StoreArgs &a, uint32_t u, uint32_t units, bool mine) : cache(-1), rows(-1) {
        if (!mine || u >= units) return;
        const uint32_t row = a.by_heads.div(u), hk = u - row * a.n_kv_heads;  // row: b * n + t
        const uint32_t b = a.by_n.div(row), t = row - b * a.n;
        rows = (int64_t)row * a.rs + (int64_t)hk * a.head_dim;
        const int p = a.pos[b];
        if (p >= 0 && (int64_t)p + a.n <= (int64_t)a.capacity)
            cache = (int64_t)b * a.cache_seq + ((int64_t)p + t) * a.cache_rs + (int64_t)hk * a.cache_head;
        else if (t == 0 && hk == 0)
            report_status(a.status, kErrBounds);
    }
    __device__ __forceinline__ int64_t cache_of(int row) const { return __shfl_sync(0xffffffffu, cache, row); }
    __device__ __forceinline__ int64_t rows_of(int row) const { return __shfl_sync(0xffffffffu, rows, row); }
};

template <typename T, int D>
__device__ __forceinline__ void fetch(const Places &at, const void *src, bool vec, Octet<T> (&x)[StoreCfg<D>::kSteps]) {
    using C = StoreCfg<D>;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int st = 0; st < C::kSteps; ++st) {
        const int it = st * 32 + lane, d = 8 * (it % C::kOcts);
        const int64_t off = at.rows_of(it / C::kOcts);
        x[st].zero();
        if (off >= 0 && d < D) x[st].load(static_cast<const T *>(src) + off + d, vec);
    }
}

template <typename T, int D, bool kIsV>
__device__ __forceinline__ void quantise(const Octet<T> (&oct)[StoreCfg<D>::kSteps], unsigned char *mine) {
    using C = StoreCfg<D>;
    using R = Q4Row<D>;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int st = 0; st < C::kSteps; ++st) {
        const int it = st * 32 + lane, row = it / C::kOcts, o = it % C::kOcts, g = o / 4, col = o & 3;
        float mn, mx, x[8];
        oct[st].ends(mn, mx);
        oct[st].get(x);
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) {
            mn = min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, off));
            mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        }
        const float range = __fsub_rn(mx, mn);
        // a NaN, an infinity or a range past the largest number has no grid: the scale is NaN
        // and so is what the group reads back as
        const bool bad = !(range <= 3.4028235e38f);
        const __nv_bfloat16 sb = __float2bfloat16_rn(__fmul_rn(range, 1.f / 15.f));
        const float s = __bfloat162float(sb);
        float z = 0.f;
        uint32_t code = 0;
        if (!bad && s > 0.f) {
            // (a scale whose reciprocal could overflow is taken 2^100 times as large, exactly)
            const float up = s < 0x1p-100f ? 0x1p100f : 1.f, div = s * up, rcp = __frcp_rn(div);
            if (up != 1.f)
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] *= up;
            const float zx[1] = {-mn * up};
            z = (float)codes_of(zx, div, rcp, 0.f);
            code = codes_of(x, div, rcp, z);
        }
        unsigned char *r = mine + row * R::kBytes;
        if (!kIsV) {
            reinterpret_cast<uint32_t *>(r)[R::k_word(g, col)] = evens_first(code);
        } else {
            // halves 2 col and 2 col + 1: byte `col` of the four lanes' codes, lane m's as nibble m.
            // A transpose of 4 x 4 bytes over the four lanes: with lane col ^ 2 the halves that hold
            // the other's bytes, then with col ^ 1 single bytes.
            const uint32_t far = __shfl_xor_sync(0xffffffffu, __byte_perm(code, 0, (col & 2) ? 0x3210 : 0x1032), 2);
            const uint32_t two = __byte_perm(code, far, (col & 2) ? 0x3254 : 0x5410);
            const uint32_t near = __shfl_xor_sync(0xffffffffu, two, 1);
            const uint32_t keep = evens_first(__byte_perm(two, near, (col & 1) ? 0x3715 : 0x6240));
            uint16_t *h = reinterpret_cast<uint16_t *>(r + R::kV) + R::v_half(g, 2 * col);
            h[0] = (uint16_t)keep;
            h[R::kSet] = (uint16_t)(keep >> 16);
        }
        if (col == 0) {
            const uint32_t lo = bad ? 0x7fc0u : (uint32_t)__bfloat16_as_ushort(sb);
            reinterpret_cast<uint32_t *>(r + (kIsV ? R::kParamV : R::kParamK))[g] =
                lo | ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(128.f + z)) << 16);
        }
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * kStoreWarps) append_q4_kernel(const Q4StoreArgs a) {
    using C = StoreCfg<D>;
    using R = Q4Row<D>;
    __shared__ __align__(16) unsigned char stage[kStoreWarps][C::kRows * R::kBytes];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t units = (uint32_t)a.batch * a.n * a.n_kv_heads;  // below 2^31
    const uint32_t u0 = (blockIdx.x * kStoreWarps + warp) * C::kRows;
    if (u0 >= units) return;
    unsigned char *mine = stage[warp];
    constexpr int kTail = (R::kBytes - R::kParamV) / 4 - R::kGroups;  // words behind the parameters
    if constexpr (kTail > 0)
        for (int i = lane; i < C::kRows * kTail; i += 32)
            *reinterpret_cast<uint32_t *>(mine + i / kTail * R::kBytes + R::kParamV + 4 * R::kGroups + 4 * (i % kTail)) = 0u;
    const Places at(a, u0 + lane, units, lane < C::kRows);
    Octet<T> k[C::kSteps], v[C::kSteps];
    fetch<T, D>(at, a.k, a.vec, k);
    fetch<T, D>(at, a.v, a.vec, v);
    quantise<T, D, false>(k, mine);
    quantise<T, D, true>(v, mine);
    __syncwarp();
#pragma unroll
    for (int p0 = 0; p0 < C::kRows * C::kPieces; p0 += 32) {
        const int p = p0 + lane, row = p / C::kPieces;
        const int64_t off = at.cache_of(min(row, C::kRows - 1));
        if (row < C::kRows && off >= 0)
            *reinterpret_cast<uint4 *>(a.cache + off + 16 * (p % C::kPieces)) = *reinterpret_cast<const uint4 *>(mine + 16 * p);
    }
}

template <typename T, int D, bool kIsV>
__device__ __forceinline__ void read_back(const Places &at, void *out, bool vec, const unsigned char *mine) {
    using C = StoreCfg<D>;
    using R = Q4Row<D>;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int st = 0; st < C::kSteps; ++st) {
        const int it = st * 32 + lane, row = it / C::kOcts, o = it % C::kOcts, g = o / 4, col = o & 3, d = 8 * o;
        const unsigned char *r = mine + row * R::kBytes;
        const uint32_t pw = reinterpret_cast<const uint32_t *>(r + (kIsV ? R::kParamV : R::kParamK))[g];
        const uint32_t bias = q4_bias2(pw), s2 = __byte_perm(pw, pw, 0x1010);
        uint32_t v[4];  // channels 2 k and 2 k + 1 as c - z
        if (!kIsV) {
            const uint32_t w = reinterpret_cast<const uint32_t *>(r)[R::k_word(g, col)];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = q4_codes2(w, k, bias);
        } else {
            const uint16_t *h = reinterpret_cast<const uint16_t *>(r + R::kV) + R::v_half(g, 2 * col);
            const uint32_t own = (uint32_t)h[0] | ((uint32_t)h[R::kSet] << 16);  // halves 2 col, 2 col + 1
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[k] = q4_codes2(__shfl_sync(0xffffffffu, own, (lane & ~3) | k), col, bias);
        }
        const int64_t off = at.rows_of(row);
        if (off >= 0 && d < D) save8(static_cast<T *>(out) + off + d, vec, v, s2);
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * kStoreWarps) expand_q4_kernel(const Q4StoreArgs a) {
    using C = StoreCfg<D>;
    using R = Q4Row<D>;
    __shared__ __align__(16) unsigned char stage[kStoreWarps][C::kRows * R::kBytes];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t units = (uint32_t)a.batch * a.n * a.n_kv_heads;
    const uint32_t u0 = (blockIdx.x * kStoreWarps + warp) * C::kRows;
    if (u0 >= units) return;
    unsigned char *mine = stage[warp];
    constexpr int kLoads = (C::kRows * C::kPieces + 31) / 32;
    Places at(a, u0 + lane, units, lane < C::kRows);
    if (at.cache < 0) at.rows = -1;  // rows left as they were
    uint4 got[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int p = lane + 32 * i, row = p / C::kPieces;
        const int64_t off = at.cache_of(min(row, C::kRows - 1));
        got[i] = make_uint4(0, 0, 0, 0);
        if (row < C::kRows && off >= 0) got[i] = *reinterpret_cast<const uint4 *>(a.cache + off + 16 * (p % C::kPieces));
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        if (lane + 32 * i < C::kRows * C::kPieces) *reinterpret_cast<uint4 *>(mine + 16 * (lane + 32 * i)) = got[i];
    __syncwarp();
    read_back<T, D, false>(at, a.k_out, a.vec, mine);
    read_back<T, D, true>(at, a.v_out, a.vec, mine);
}

template <typename T, int D>
cudaError_t launch_store_td(const Q4StoreArgs &a, bool expand, cudaStream_t s) {
    const int64_t units = (int64_t)a.batch * a.n * a.n_kv_heads;
    constexpr int kPer = kStoreWarps * StoreCfg<D>::kRows;
    const int64_t blocks = (units + kPer - 1) / kPer;
    if (blocks == 0) return cudaSuccess;
    if (expand)
        expand_q4_kernel<T, D><<<(unsigned)blocks, 32 * kStoreWarps, 0, s>>>(a);
    else
        append_q4_kernel<T, D><<<(unsigned)blocks, 32 * kStoreWarps, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_store_t(const Q4StoreArgs &a, bool expand, cudaStream_t s) {
    switch (a.head_dim) {
        case 64: return launch_store_td<T, 64>(a, expand, s);
        case 80: return launch_store_td<T, 80>(a, expand, s);
        case 128: return launch_store_td<T, 128>(a, expand, s);
        case 256: return launch_store_td<T, 256>(a, expand, s);
        case 512: return launch_store_td<T, 512>(a, expand, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

int q4_row_bytes(int head_dim) {
    switch (head_dim) {
        case 64: return Q4Row<64>::kBytes;
        case 80: return Q4Row<80>::kBytes;
        case 128: return Q4Row<128>::kBytes;
        case 256: return Q4Row<256>::kBytes;
        case 512: return Q4Row<512>::kBytes;
        default: return 0;
    }
}

cudaError_t launch_q4_store(const Q4StoreArgs &a, bool bf16, bool expand, cudaStream_t s) {
    return bf16 ? launch_store_t<__nv_bfloat16>(a, expand, s) : launch_store_t<float>(a, expand, s);
}

}  // namespace lat
