// split_join.cuh — joins the partial results of a split-KV decode.
//
// The pieces of one (sequence, query head) hold normalised outputs o_c and log2-domain
// log-sum-exps lse_c over disjoint keys, so
//   lse = log2 sum_c 2^{lse_c},   out = sum_c 2^{lse_c - lse} o_c
// (a piece without keys has lse_c = -inf and counts for nothing).  A CTA of four warps takes up
// to 128 channels of one head; warp w takes pieces w, w + 4, ..., four in flight at a time.
// It waits for the grid before it (a programmatic dependent launch), so its own start is hidden.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.cuh"

namespace lat {

struct JoinArgs {
    const float *part_o;         // [batch, n_heads, max_splits, head_dim]
    const float *part_lse;       // [batch, n_heads, max_splits]
    const int32_t *piece_count;  // [batch, n_heads]; 0 or 1: nothing to join
    int max_splits, n_heads;
    void *out;
    int64_t out_rs;
    float *lse;
};

constexpr int kJoinWarps = 4;

template <int D, bool F32>
__global__ void __launch_bounds__(32 * kJoinWarps) split_join_kernel(const JoinArgs a) {
    constexpr int kW = D < 128 ? D : 128, kV4 = kW / 4, kCols = (D + kW - 1) / kW;
    __shared__ float4 part[kJoinWarps][32];
    __shared__ float sm[kJoinWarps], sz[kJoinWarps];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t bh = blockIdx.x / kCols;
    const int nseg = min(a.piece_count[bh], a.max_splits);
    if (nseg <= 1) return;  // written whole
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x % kCols * kV4 + lane;
    const float *pl = a.part_lse + bh * a.max_splits;
    const float4 *po = reinterpret_cast<const float4 *>(a.part_o + bh * a.max_splits * D) + col;
    float m = -INFINITY, z = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = warp; s0 < nseg; s0 += 4 * kJoinWarps) {
        float l[4];
        float4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int s = s0 + k * kJoinWarps;
            l[k] = s < nseg ? __ldcg(pl + s) : -INFINITY;
            v[k] = s < nseg && lane < kV4 ? __ldcg(po + (int64_t)s * (D / 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float mn = m;
#pragma unroll
        for (int k = 0; k < 4; ++k) mn = fmaxf(mn, l[k]);
        const float base = mn == -INFINITY ? 0.f : mn, cf = fast_exp2(m - base);
        z *= cf; o.x *= cf; o.y *= cf; o.z *= cf; o.w *= cf;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float w = fast_exp2(l[k] - base);
            z += w;
            o.x = fmaf(w, v[k].x, o.x); o.y = fmaf(w, v[k].y, o.y);
            o.z = fmaf(w, v[k].z, o.z); o.w = fmaf(w, v[k].w, o.w);
        }
        m = mn;
    }
    part[warp][lane] = o;
    if (lane == 0) sm[warp] = m, sz[warp] = z;
    __syncthreads();
    if (warp != 0) return;
    float M = sm[0], Z = 0.f;
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) M = fmaxf(M, sm[w]);
    const float base = M == -INFINITY ? 0.f : M;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        const float f = fast_exp2(sm[w] - base);
        const float4 v = part[w][lane];
        Z = fmaf(f, sz[w], Z);
        o.x = fmaf(f, v.x, o.x); o.y = fmaf(f, v.y, o.y); o.z = fmaf(f, v.z, o.z); o.w = fmaf(f, v.w, o.w);
    }
    const float rz = Z == 0.f ? 0.f : 1.f / Z;
    if (lane < kV4) {
        const int64_t b = bh / a.n_heads, h = bh % a.n_heads, at = b * a.out_rs + h * D + 4 * col;
        if constexpr (F32)
            *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = make_float4(o.x * rz, o.y * rz, o.z * rz, o.w * rz);
        else
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + at) =
                make_uint2(pack_bf16x2(o.x * rz, o.y * rz), pack_bf16x2(o.z * rz, o.w * rz));
    }
    if (blockIdx.x % kCols == 0 && lane == 0 && a.lse != nullptr)
        a.lse[bh] = (M + log2f(Z)) * 0.69314718055994531f;  // log2f(0) is -inf
}

// `rows` = batch * n_heads; the launch before it on the stream writes the pieces
template <int D, bool F32>
cudaError_t launch_split_join(const JoinArgs &a, int64_t rows, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(rows * ((D + 127) / 128)));
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, split_join_kernel<D, F32>, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace lat
