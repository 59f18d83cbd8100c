// kv_q4.cu — rows into and out of the 4-bit KV cache (the row format: q4_row.cuh).
//
// Append: rows pos[b] + t of sequence b's cache take the quantised new rows (t < n_new).
// Expand: rows pos[b] + t read back as K and V rows.  Both move bytes: 4 bytes a channel of
// bf16 K and V on one side, 1.25 on the other.
//
// How: a warp takes kRows head rows at once, so that their loads are in flight together.  A
// lane works on 8 neighbouring channels (an octet: one 16-byte vector of bf16), four lanes
// on a group.  K's octet is one word of the row; V's octet is one nibble of eight halves, so
// the four lanes of a group OR their nibbles together.  Packed rows pass through shared
// memory, so that the cache is read and written in 16-byte vectors.  Every step of the
// quantisation is one fp32 operation rounded to nearest, the same on any machine.
#include <math.h>

#include "device_common.cuh"
#include "kernels.h"
#include "q4_row.cuh"

namespace lat {

namespace {

constexpr int kStoreWarps = 4;

template <typename T>
__device__ __forceinline__ void load8(const T *p, bool vec, float x[8]);
template <>
__device__ __forceinline__ void load8<float>(const float *p, bool vec, float x[8]) {
    if (vec) {
        const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = p[k];
    }
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16 *p, bool vec, float x[8]) {
    if (vec) {
        const uint4 a = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[2 * k] = __uint_as_float(w[k] << 16);
            x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = __bfloat162float(p[k]);
    }
}

template <typename T>
__device__ __forceinline__ void save8(T *p, bool vec, const float x[8]);
template <>
__device__ __forceinline__ void save8<float>(float *p, bool vec, const float x[8]) {
    if (vec) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) p[k] = x[k];
    }
}
template <>
__device__ __forceinline__ void save8<__nv_bfloat16>(__nv_bfloat16 *p, bool vec, const float x[8]) {
    if (vec) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                   pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) p[k] = __float2bfloat16_rn(x[k]);
    }
}

// The whole number nearest to x / s, ties to even, exactly: n = rint(x * (1 / s)) is within one
// of it, and the remainder x - n s is exact in fp32 (s has 8 bits; for n = 0 it is x, and for
// n != 0 it ends no lower than x's last place and stays below 2 s).
__device__ __forceinline__ float round_quotient(float x, float s, float r) {
    float n = rintf(x * r);
    const float twice = 2.f * fmaf(-n, s, x);
    const bool odd = ((int)n & 1) != 0;
    if (twice > s || (twice == s && odd)) n += 1.f;
    else if (twice < -s || (twice == -s && odd)) n -= 1.f;
    return n;
}

template <int D>
struct StoreCfg {
    using R = Q4Row<D>;
    static constexpr int kRows = D <= 80 ? 4 : (D == 128 ? 4 : (D == 256 ? 2 : 1));  // a warp's head rows
    static constexpr int kOcts = R::kPad / 4;       // octets of a head row, K's then V's
    static constexpr int kSteps = kRows * kOcts / 32;
    static_assert(kRows * kOcts % 32 == 0, "every lane has an octet in every step");
    static constexpr int kChunks = kRows * R::kBytes / 16;  // 16-byte pieces of the packed rows
};

// head row `u` (of batch * n * n_kv_heads) -> its sequence, row and head; false when it is
// past the end or its sequence does not fit the cache (reported once per sequence)
__device__ __forceinline__ bool locate(const Q4StoreArgs &a, uint32_t u, uint32_t units, int64_t *slot) {
    if (u >= units) return false;
    const uint32_t r = u / a.n_kv_heads, hk = u - r * a.n_kv_heads;
    const uint32_t b = r / a.n, t = r - b * a.n;
    const int p = a.pos[b];
    if (p < 0 || (int64_t)p + a.n > (int64_t)a.capacity) {
        if (t == 0 && hk == 0) report_status(a.status, kErrBounds);
        return false;
    }
    *slot = (int64_t)b * a.cache_seq + ((int64_t)p + t) * a.cache_rs + (int64_t)hk * a.cache_head;
    return true;
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

    int64_t slot[C::kRows];
    bool live[C::kRows];
#pragma unroll
    for (int i = 0; i < C::kRows; ++i) live[i] = locate(a, u0 + i, units, &slot[i]);

    float x[C::kSteps][8];
#pragma unroll
    for (int st = 0; st < C::kSteps; ++st) {
        const int it = st * 32 + lane, row = it / C::kOcts, o = it % C::kOcts;
        const int d = 8 * (o % (C::kOcts / 2));
        const bool is_v = o >= C::kOcts / 2;
#pragma unroll
        for (int k = 0; k < 8; ++k) x[st][k] = 0.f;
        const uint32_t u = u0 + row, ur = u / a.n_kv_heads;
        if (u < units && d < D) {
            const T *src = static_cast<const T *>(is_v ? a.v : a.k) + (int64_t)ur * a.rs + (u - ur * a.n_kv_heads) * D + d;
            load8<T>(src, a.vec, x[st]);
        }
    }
    // the padding behind the parameters
    if (R::kParamV + 4 * R::kGroups < R::kBytes)
        for (int i = lane; i < C::kRows * ((R::kBytes - R::kParamV) / 4 - R::kGroups); i += 32) {
            constexpr int kW = (R::kBytes - R::kParamV) / 4 - R::kGroups > 0
                                   ? (R::kBytes - R::kParamV) / 4 - R::kGroups : 1;
            *reinterpret_cast<uint32_t *>(mine + i / kW * R::kBytes + R::kParamV + 4 * R::kGroups + 4 * (i % kW)) = 0u;
        }
#pragma unroll
    for (int st = 0; st < C::kSteps; ++st) {
        const int it = st * 32 + lane, row = it / C::kOcts, o = it % C::kOcts;
        const bool is_v = o >= C::kOcts / 2;
        const int g = o % (C::kOcts / 2) / 4, col = o & 3;
        float mn = 0.f, mx = 0.f;
        bool bad = false;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            mn = fminf(mn, x[st][k]);
            mx = fmaxf(mx, x[st][k]);
            bad |= x[st][k] != x[st][k];
        }
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) {
            mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            bad |= __shfl_xor_sync(0xffffffffu, (int)bad, off) != 0;
        }
        const float range = __fsub_rn(mx, mn);
        // a NaN, an infinity or a range past the largest number has no grid: the scale is NaN
        // and so is what the group reads back as
        bad |= !(range <= 3.4028235e38f);
        __nv_bfloat16 sb = __float2bfloat16_rn(__fmul_rn(range, 1.f / 15.f));
        const float s = __bfloat162float(sb);
        const bool flat = bad || !(s > 0.f);
        // (a scale whose reciprocal could overflow is taken 2^100 times as large, exactly)
        const float up = flat ? 0.f : (s < 0x1p-100f ? 0x1p100f : 1.f);
        const float div = flat ? 1.f : s * up, rcp = __frcp_rn(div);
        const float z = flat ? 0.f : fminf(fmaxf(round_quotient(-mn * up, div, rcp), 0.f), 15.f);
        uint32_t code = 0;  // 8 codes, channel k at nibble k
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float c = flat ? 0.f : fminf(fmaxf(round_quotient(x[st][k] * up, div, rcp) + z, 0.f), 15.f);
            code |= (uint32_t)c << (4 * k);
        }
        // V: halves 2m and 2m + 1 take this lane's codes 2m and 2m + 1 as nibble `col`
        uint32_t vw[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            vw[m] = (((code >> (8 * m)) & 15u) << (4 * col)) | (((code >> (8 * m + 4)) & 15u) << (16 + 4 * col));
            vw[m] |= __shfl_xor_sync(0xffffffffu, vw[m], 1);
            vw[m] |= __shfl_xor_sync(0xffffffffu, vw[m], 2);
        }
        {
            unsigned char *r = mine + row * R::kBytes;
            const int off = (g / R::kSet * 4 + col) * R::kSet + g % R::kSet;
            if (!is_v) {
                uint32_t w = 0;  // nibble i holds channel 2 i, nibble i + 4 channel 2 i + 1
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w |= (((code >> (8 * i)) & 15u) << (4 * i)) | (((code >> (8 * i + 4)) & 15u) << (16 + 4 * i));
                reinterpret_cast<uint32_t *>(r)[off] = w;
            } else {
                const uint32_t w = col == 0 ? vw[0] : col == 1 ? vw[1] : col == 2 ? vw[2] : vw[3];
                uint16_t *h = reinterpret_cast<uint16_t *>(r + R::kV) + (g / R::kSet * 8 + 2 * col) * R::kSet + g % R::kSet;
                h[0] = (uint16_t)w;
                h[R::kSet] = (uint16_t)(w >> 16);
            }
            if (col == 0) {
                const uint32_t lo = bad ? 0x7fc0u : (uint32_t)__bfloat16_as_ushort(sb);
                reinterpret_cast<uint32_t *>(r + (is_v ? R::kParamV : R::kParamK))[g] =
                    lo | ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(128.f + z)) << 16);
            }
        }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < C::kRows; ++i)
        if (live[i])
            for (int c = lane; c < R::kBytes / 16; c += 32)
                *reinterpret_cast<uint4 *>(a.cache + slot[i] + 16 * c) =
                    *reinterpret_cast<const uint4 *>(mine + i * R::kBytes + 16 * c);
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * kStoreWarps) expand_q4_kernel(const Q4StoreArgs a) {
    using C = StoreCfg<D>;
    using R = Q4Row<D>;
    __shared__ __align__(16) unsigned char stage[kStoreWarps][C::kRows * R::kBytes];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t units = (uint32_t)a.batch * a.n * a.n_kv_heads;  // below 2^31
    const uint32_t u0 = (blockIdx.x * kStoreWarps + warp) * C::kRows;
    if (u0 >= units) return;
    unsigned char *mine = stage[warp];
    constexpr int kPieces = R::kBytes / 16, kLoads = (C::kChunks + 31) / 32;
    uint4 got[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int p = lane + 32 * i, row = p / kPieces;
        int64_t slot;
        got[i] = make_uint4(0, 0, 0, 0);
        if (row < C::kRows && locate(a, u0 + row, units, &slot))
            got[i] = *reinterpret_cast<const uint4 *>(a.cache + slot + 16 * (p % kPieces));
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int p = lane + 32 * i;
        if (p < C::kChunks) *reinterpret_cast<uint4 *>(mine + 16 * p) = got[i];
    }
    __syncwarp();
#pragma unroll
    for (int st = 0; st < C::kSteps; ++st) {
        const int it = st * 32 + lane, row = it / C::kOcts, o = it % C::kOcts;
        const bool is_v = o >= C::kOcts / 2;
        const int g = o % (C::kOcts / 2) / 4, col = o & 3, d = 8 * (o % (C::kOcts / 2));
        const uint32_t u = u0 + row, ur = u / a.n_kv_heads;
        if (u >= units || d >= D) continue;
        const int p0 = a.pos[ur / a.n];
        if (p0 < 0 || (int64_t)p0 + a.n > (int64_t)a.capacity) continue;  // rows left as they were
        const unsigned char *r = mine + row * R::kBytes;
        uint32_t code = 0;  // channel k at nibble k
        if (!is_v) {
            const uint32_t w = reinterpret_cast<const uint32_t *>(r)[(g / R::kSet * 4 + col) * R::kSet + g % R::kSet];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                code |= (((w >> (4 * i)) & 15u) << (8 * i)) | (((w >> (16 + 4 * i)) & 15u) << (8 * i + 4));
        } else {
            const uint16_t *h = reinterpret_cast<const uint16_t *>(r + R::kV) + g / R::kSet * 8 * R::kSet + g % R::kSet;
#pragma unroll
            for (int k = 0; k < 8; ++k) code |= (((uint32_t)h[k * R::kSet] >> (4 * col)) & 15u) << (4 * k);
        }
        const uint32_t pw = reinterpret_cast<const uint32_t *>(r + (is_v ? R::kParamV : R::kParamK))[g];
        const float s = q4_scale(pw), z = __uint_as_float(pw & 0xffff0000u) - 128.f;
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = s * ((float)((code >> (4 * k)) & 15u) - z);
        T *dst = static_cast<T *>(is_v ? a.v_out : a.k_out) + (int64_t)ur * a.rs + (u - ur * a.n_kv_heads) * D + d;
        save8<T>(dst, a.vec, x);
    }
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
