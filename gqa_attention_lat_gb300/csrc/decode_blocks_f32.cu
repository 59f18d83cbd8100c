// decode_blocks_f32.cu — fp32 decode over chosen blocks of an in-place cache.
//
// For each sequence and KV head the query heads attend to the keys of the listed blocks
// (block_select.cu makes such lists), in fp32 on the CUDA cores, whose products lose nothing.
//
// How: CTA (unit, piece): a unit is one sequence, one KV head and up to 4 of its query heads, so
// that a key is loaded once for all of them; its listed keys are cut into `splits` pieces, joined
// by split_join.cuh.  A warp takes kKeys keys at a time, a lane 4 neighbouring channels of every
// 128.  The kKeys * 4 scores come out of the lanes' partial sums by a butterfly that halves the
// values at every step (31 shuffles for 32 scores instead of 160), one score a lane; the weights
// go back by a shuffle each.  Bound by the bytes of K and V where many pieces are in flight, by
// the loads' round trips where few are.
#include <math.h>

#include <algorithm>

#include "cache_kernels.h"
#include "device_common.cuh"
#include "split_join.cuh"

namespace lat {

namespace {

constexpr int kBWarps = 4;
constexpr int kBHeads = 4;
// keys a piece is worth (one sequence, 2 KV heads of 8 query heads, head_dim 256: 2048 listed keys
// 13.3 us at 16, 9.5 at 32, 9.3 at 64, 11.7 at 128; 256 of them 5.4, 6.0, 7.6, 10.9)
constexpr int kMinKeys = 64;

template <int D>
__global__ void __launch_bounds__(32 * kBWarps) decode_blocks_f32_kernel(const BlocksF32Args a) {
    constexpr int NT = (D + 127) / 128;                     // 16-byte vectors a lane and row
    constexpr int kKeys = NT == 1 ? 8 : (NT == 2 ? 4 : 2);  // keys at a time
    constexpr int N = kKeys * kBHeads;                      // scores at a time
    constexpr int kLow = N == 32 ? 0 : (N == 16 ? 1 : 2);   // lane bits below a score's place
    __shared__ float4 part[kBWarps][kBHeads][NT][32];
    __shared__ float sm[kBWarps][kBHeads], sl[kBWarps][kBHeads];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = a.n_heads / a.n_kv_heads, HB = (G + kBHeads - 1) / kBHeads;
    const int piece = blockIdx.x % a.splits;
    const int64_t unit = blockIdx.x / a.splits;
    const int hb = (int)(unit % HB), hk = (int)(unit / HB % a.n_kv_heads), b = (int)(unit / HB / a.n_kv_heads);
    const int h0 = hk * G + hb * kBHeads, heads = min(kBHeads, G - hb * kBHeads);
    const int64_t bh0 = (int64_t)b * a.n_heads + h0;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int len = a.kv_lens[b];
    const bool bad = len < 0 || len > a.max_kv_len;
    if (threadIdx.x < heads && piece == 0 && a.splits > 1) a.piece_count[bh0 + threadIdx.x] = bad ? 0 : a.splits;
    if (bad) {
        if (threadIdx.x == 0 && piece == 0 && hk == 0 && hb == 0) report_status(a.status, kErrBounds);
        return;
    }
    float4 q[kBHeads][NT], o[kBHeads][NT];
#pragma unroll
    for (int h = 0; h < kBHeads; ++h)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int d = 4 * lane + 128 * t;
            const bool live = h < heads && d < D;
            q[h][t] = live ? *reinterpret_cast<const float4 *>(a.q + (int64_t)b * a.q_rs + (int64_t)(h0 + h) * D + d)
                           : make_float4(0.f, 0.f, 0.f, 0.f);
            o[h][t] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    const float *kb = a.k + (int64_t)b * a.cache_seq + (int64_t)hk * a.cache_head + 4 * lane;
    const float *vb = a.v + (int64_t)b * a.cache_seq + (int64_t)hk * a.cache_head + 4 * lane;
    const int32_t *list = a.blocks + ((int64_t)b * a.n_kv_heads + hk) * a.n_sel;
    const int nblk = len == 0 ? 0 : (len - 1) / a.block_size + 1, slots = min(a.n_sel, nblk);
    const int steps = slots * (a.block_size / kKeys);  // of kKeys keys, block after block
    const int per = (steps + a.splits - 1) / a.splits;
    const int end = min(steps, (piece + 1) * per);
    const int me = lane >> kLow, my_head = me % kBHeads, my_key = me / kBHeads;
    float m = -INFINITY, l = 0.f;  // of this lane's head
    for (int s = piece * per + warp; s < end; s += kBWarps) {
        const int slot = s / (a.block_size / kKeys);
        const int blk = list[slot], before = slot > 0 ? list[slot - 1] : -1;
        const bool fits = blk >= 0 && blk < nblk && (slot == 0 || (before >= 0 && before < blk));
        if (!fits) {  // -1 is padding
            if (blk != -1 && lane == 0) report_status(a.status, kErrBounds);
            continue;
        }
        const int j0 = blk * a.block_size + s % (a.block_size / kKeys) * kKeys;
        const int n = min(kKeys, len - j0);
        if (n <= 0) continue;
        float4 kx[kKeys][NT], vx[kKeys][NT];
#pragma unroll
        for (int u = 0; u < kKeys; ++u)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const bool live = u < n && 4 * lane + 128 * t < D;
                const int64_t at = (int64_t)(j0 + u) * a.cache_rs + 128 * t;
                kx[u][t] = live ? *reinterpret_cast<const float4 *>(kb + at) : make_float4(0.f, 0.f, 0.f, 0.f);
                vx[u][t] = live ? *reinterpret_cast<const float4 *>(vb + at) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        float x[N];
#pragma unroll
        for (int u = 0; u < kKeys; ++u)
#pragma unroll
            for (int h = 0; h < kBHeads; ++h) {
                float p = 0.f;
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    p = fmaf(q[h][t].x, kx[u][t].x, fmaf(q[h][t].y, kx[u][t].y, fmaf(q[h][t].z, kx[u][t].z, fmaf(q[h][t].w, kx[u][t].w, p))));
                x[u * kBHeads + h] = p;
            }
        int off = 16;
#pragma unroll
        for (int half = N / 2; half >= 1; half /= 2, off /= 2) {
            const bool up = lane & off;
#pragma unroll
            for (int i = 0; i < half; ++i) {
                const float keep = up ? x[i + half] : x[i], send = up ? x[i] : x[i + half];
                x[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
            }
        }
#pragma unroll
        for (int k = kLow - 1; k >= 0; --k) x[0] += __shfl_xor_sync(0xffffffffu, x[0], 1 << k);
        float sc = a.cap_log2 > 0.f ? a.cap_log2 * tanhf(x[0] * a.raw_over_cap) : x[0] * a.scale_log2;
        if (my_key >= n) sc = -INFINITY;
        float top = sc;
#pragma unroll
        for (int k = 4 << kLow; k < 32; k *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
        const float m_new = fmaxf(m, top);
        const float base = m_new == -INFINITY ? 0.f : m_new;
        const float corr = fast_exp2(m - base), p = fast_exp2(sc - base);
        l = l * corr + p;  // this lane's keys only; the lanes of a head meet at the end
        m = m_new;
#pragma unroll
        for (int h = 0; h < kBHeads; ++h) {
            const float cf = __shfl_sync(0xffffffffu, corr, h << kLow);
            float w[kKeys];
#pragma unroll
            for (int u = 0; u < kKeys; ++u) w[u] = __shfl_sync(0xffffffffu, p, (u * kBHeads + h) << kLow);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float4 y = o[h][t];
                y.x *= cf; y.y *= cf; y.z *= cf; y.w *= cf;
#pragma unroll
                for (int u = 0; u < kKeys; ++u) {
                    y.x = fmaf(w[u], vx[u][t].x, y.x); y.y = fmaf(w[u], vx[u][t].y, y.y);
                    y.z = fmaf(w[u], vx[u][t].z, y.z); y.w = fmaf(w[u], vx[u][t].w, y.w);
                }
                o[h][t] = y;
            }
        }
    }
#pragma unroll
    for (int k = 4 << kLow; k < 32; k *= 2) l += __shfl_xor_sync(0xffffffffu, l, k);
    if (lane < (4 << kLow) && (lane & ((1 << kLow) - 1)) == 0) sm[warp][my_head] = m, sl[warp][my_head] = l;
#pragma unroll
    for (int h = 0; h < kBHeads; ++h)
#pragma unroll
        for (int t = 0; t < NT; ++t) part[warp][h][t][lane] = o[h][t];
    __syncthreads();
    for (int i = threadIdx.x; i < heads * NT * 32; i += 32 * kBWarps) {
        const int h = i / (NT * 32), t = i / 32 % NT, d = 4 * (i & 31) + 128 * t;
        if (d >= D) continue;
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < kBWarps; ++w) M = fmaxf(M, sm[w][h]);
        const float base = M == -INFINITY ? 0.f : M;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kBWarps; ++w) {
            const float f = fast_exp2(sm[w][h] - base);
            const float4 v = part[w][h][t][i & 31];
            L = fmaf(f, sl[w][h], L);
            y.x = fmaf(f, v.x, y.x); y.y = fmaf(f, v.y, y.y); y.z = fmaf(f, v.z, y.z); y.w = fmaf(f, v.w, y.w);
        }
        const float rl = L == 0.f ? 0.f : 1.f / L;  // 0: no listed key is there
        y.x *= rl; y.y *= rl; y.z *= rl; y.w *= rl;
        const float lse2 = M + log2f(L);
        if (a.splits == 1) {
            *reinterpret_cast<float4 *>(a.out + (int64_t)b * a.out_rs + (int64_t)(h0 + h) * D + d) = y;
            if (d == 0 && a.lse != nullptr) a.lse[bh0 + h] = lse2 * 0.69314718055994531f;
        } else {
            const int64_t at = (bh0 + h) * a.splits + piece;
            *reinterpret_cast<float4 *>(a.part_o + at * D + d) = y;
            if (d == 0) a.part_lse[at] = lse2;
        }
    }
}

template <int D>
cudaError_t launch_d(const BlocksF32Args &a, unsigned grid, cudaStream_t s) {
    decode_blocks_f32_kernel<D><<<grid, 32 * kBWarps, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || a.splits == 1) return e;
    const JoinArgs j{a.part_o, a.part_lse, a.piece_count, a.splits, a.n_heads, a.out, a.out_rs, a.lse};
    return launch_split_join<D, true>(j, (int64_t)a.batch * a.n_heads, s);
}

}  // namespace

int blocks_f32_splits(int batch, int n_heads, int n_kv_heads, int block_size, int n_sel, int num_sms) {
    const int G = n_heads / n_kv_heads;
    const int64_t units = std::max<int64_t>(1, (int64_t)batch * n_kv_heads * ((G + kBHeads - 1) / kBHeads));
    const int64_t keys = (int64_t)n_sel * block_size;
    const int64_t want = (6 * (int64_t)num_sms + units - 1) / units;  // six CTAs an SM
    return (int)std::max<int64_t>(1, std::min(want, keys / kMinKeys));
}

cudaError_t launch_decode_blocks_f32(const BlocksF32Args &a, cudaStream_t s) {
    const int G = a.n_heads / a.n_kv_heads;
    const int64_t grid = (int64_t)a.batch * a.n_kv_heads * ((G + kBHeads - 1) / kBHeads) * a.splits;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    switch (a.head_dim) {
        case 64: return launch_d<64>(a, (unsigned)grid, s);
        case 80: return launch_d<80>(a, (unsigned)grid, s);
        case 128: return launch_d<128>(a, (unsigned)grid, s);
        case 256: return launch_d<256>(a, (unsigned)grid, s);
        case 512: return launch_d<512>(a, (unsigned)grid, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace lat
