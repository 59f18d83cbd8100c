// evict.cu — the cached keys of each KV head that stay, by the attention weight they were given,
// and their rows moved up in place.
//
// choose: a cluster of up to eight CTAs takes one (sequence, KV head).  Each CTA reads its slice of
// the weights once, into shared memory; what follows runs there.  The n-th largest weight is found
// digit by digit (11, 11 and 10 bits of an order-preserving integer), counting a digit's keys into
// 2048 bins that the cluster adds up through distributed shared memory.  Then a key stays if it is
// among the first or the last, is above that weight, or equals it and few equal ones come before it;
// ballots and a scan over warps and CTAs give its place, so lists are ascending, ties go to the
// lowest key, and nothing depends on an order of execution.  Since the weights wait in shared memory,
// they may be written over the ones they came from.
// What bounds it: barriers and round trips within the cluster, then HBM (4 bytes a key).
//
// rows: row i of a head becomes its row kept[i] >= i, for ascending i.  A cluster takes K or V of one
// (sequence, KV head) and moves a stretch of rows at a time: asynchronous copies bring them to shared
// memory some stretches ahead, and a stretch is written only after the whole cluster has it.  That
// is all the order that is needed: what a stretch writes lies before every row that a later one
// reads.  Rows that stay where they are are not touched.
// What bounds it: HBM, rows read and written once.
#include "cache_kernels.h"
#include "device_common.cuh"

namespace lat {

namespace {

// ---------------------------------------------------------------------------------- choose
constexpr int kChooseThreads = 512, kChooseWarps = kChooseThreads / 32;
constexpr int kBins = 2048;
// keys a CTA takes before the cluster grows (64 heads of 65536 keys: 4096 16.0 us, 8192 .. us)
constexpr int kSliceWanted = 4096;

// order-preserving: larger weights to larger integers, NaN above all, -0 as 0
__device__ __forceinline__ uint32_t ordered(float f) {
    if (f != f) return 0xffffffffu;
    const uint32_t b = __float_as_uint(f + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint32_t load_cluster(const void *p, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(p, rank)) : "memory");
    return v;
}
// the sum of x over the CTA's threads before this one; `warps` in shared memory
__device__ __forceinline__ int scan_before(int x, int *warps) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
    }
    __syncthreads();
    if (lane == 31) warps[warp] = incl;
    __syncthreads();
    int before = incl - x;
    for (int w = 0; w < warp; ++w) before += warps[w];
    return before;
}

struct Choose {  // in shared memory, one a CTA
    uint32_t bins[kBins];
    int warps[kChooseWarps];
    int ties[kChooseWarps], sure[kChooseWarps];  // by warp
    int all_ties, all_sure;
    uint32_t digit;
    int above;       // keys in the digits above
};

__global__ void __launch_bounds__(kChooseThreads) evict_choose_kernel(const EvictChooseArgs a) {
    extern __shared__ __align__(16) unsigned char raw[];
    Choose &sh = *reinterpret_cast<Choose *>(raw);
    float *held = reinterpret_cast<float *>(raw + sizeof(Choose));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P = a.cluster, rank = (int)(blockIdx.x % P);
    const int64_t unit = blockIdx.x / P;
    const int b = (int)(unit / a.n_kv_heads), hk = (int)(unit % a.n_kv_heads);
    const int len = a.kv_lens[b];
    int32_t *kept = a.kept + unit * a.n_keep;
    const float *w = a.weights + (int64_t)b * a.w_seq + (int64_t)hk * a.w_head;
    float *out = a.out == nullptr ? nullptr : a.out + (int64_t)b * a.out_seq + (int64_t)hk * a.out_head;
    if (len < 0 || len > a.max_kv_len) {  // (the whole cluster alike)
        if (hk == 0 && rank == 0 && tid == 0) report_status(a.status, kErrBounds);
        return;
    }
    if (hk == 0 && rank == 0 && tid == 0) a.new_lens[b] = min(len, a.n_keep);
    if (len <= a.n_keep) {  // everything stays
        for (int i = rank * kChooseThreads + tid; i < a.n_keep; i += P * kChooseThreads) kept[i] = i < len ? i : -1;
        if (out != nullptr && out != w)
            for (int i = rank * kChooseThreads + tid; i < len; i += P * kChooseThreads) out[i] = w[i];
        return;
    }
    // ---- this CTA's slice ------------------------------------------------------------------
    const int slice = (len + P - 1) / P, lo = min(len, rank * slice), n = min(len, lo + slice) - lo;
    const int mid_lo = a.n_first, mid_hi = len - a.n_last;  // keys that are chosen among
    for (int i = tid; i < n; i += kChooseThreads) held[i] = __ldcg(w + lo + i);  // (they may be written over)
    auto chosen_among = [&](int i) { return lo + i >= mid_lo && lo + i < mid_hi; };

    // ---- the weight that the last chosen key has, digit by digit ---------------------------------
    int need = a.n_keep - a.n_first - a.n_last;  // keys still to be chosen among those with the prefix
    uint32_t prefix = 0, mask = 0;
    if (need > 0) {
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
            for (int i = tid; i < kBins; i += kChooseThreads) sh.bins[i] = 0;
            __syncthreads();
            for (int i = tid; i < n; i += kChooseThreads) {
                const uint32_t k = ordered(held[i]);
                if ((k & mask) == prefix && chosen_among(i)) atomicAdd(&sh.bins[(k >> shift) & ((1u << bits) - 1)], 1u);
            }
            if (P > 1) cluster_sync_all();
            else __syncthreads();
            // the cluster's counts, largest digits first: thread t has four, and what lies above
            uint32_t c[4];
            int mine = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int bin = kBins - 1 - (4 * tid + q);
                c[q] = sh.bins[bin];
                for (int p = 1; p < P; ++p) c[q] += load_cluster(&sh.bins[bin], (uint32_t)((rank + p) % P));
                mine += (int)c[q];
            }
            int above = scan_before(mine, sh.warps);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (above < need && above + (int)c[q] >= need) sh.digit = kBins - 1 - (4 * tid + q), sh.above = above;
                above += (int)c[q];
            }
            if (P > 1) cluster_sync_all();  // (also: the bins have been read)
            else __syncthreads();
            prefix |= sh.digit << shift;
            mask |= ((1u << bits) - 1) << shift;
            need -= sh.above;
            __syncthreads();
        }
    } else {
        mask = 0xffffffffu, prefix = 0xffffffffu;  // (NaN would tie; `need` 0 keeps none)
    }
    // ---- places: a warp takes a run of the slice, in order ------------------------------------------
    // (a key of rank: 2 stays, 1 is one of the equal ones, 0 goes)
    auto rank_of = [&](int i) {
        if (i >= n) return 0;
        if (!chosen_among(i)) return 2;
        if (a.n_keep == a.n_first + a.n_last) return 0;
        const uint32_t k = ordered(held[i]);
        return k > prefix ? 2 : k == prefix ? 1 : 0;
    };
    const int run = (slice + kChooseWarps * 32 - 1) / (kChooseWarps * 32) * 32;  // keys of a warp
    int ties = 0, sure = 0;
    for (int i0 = warp * run; i0 < (warp + 1) * run; i0 += 32) {
        const int r = rank_of(i0 + lane);
        ties += __popc(__ballot_sync(0xffffffffu, r == 1));
        sure += __popc(__ballot_sync(0xffffffffu, r == 2));
    }
    if (lane == 0) sh.ties[warp] = ties, sh.sure[warp] = sure;
    __syncthreads();
    if (tid == 0) {
        int t = 0, s = 0;
        for (int x = 0; x < kChooseWarps; ++x) {
            const int ti = sh.ties[x], si = sh.sure[x];
            sh.ties[x] = t, sh.sure[x] = s;
            t += ti, s += si;
        }
        sh.all_ties = t, sh.all_sure = s;
    }
    if (P > 1) cluster_sync_all();
    else __syncthreads();
    int ties_before = sh.ties[warp], sure_before = sh.sure[warp];
    for (int p = 0; p < rank; ++p) {
        ties_before += (int)load_cluster(&sh.all_ties, (uint32_t)p);
        sure_before += (int)load_cluster(&sh.all_sure, (uint32_t)p);
    }
    const uint32_t under = (1u << lane) - 1;
    for (int i0 = warp * run; i0 < (warp + 1) * run; i0 += 32) {
        const int i = i0 + lane, r = rank_of(i);
        const uint32_t tied = __ballot_sync(0xffffffffu, r == 1);
        const int t = ties_before + __popc(tied & under);  // equal ones before this key
        const uint32_t stay = __ballot_sync(0xffffffffu, r == 2);
        if (r == 2 || (r == 1 && t < need)) {
            // sure ones before, and the equal ones before that stay
            const int at = sure_before + __popc(stay & under) + min(t, need);
            kept[at] = lo + i;
            if (out != nullptr) out[at] = held[i];
        }
        ties_before += __popc(tied);
        sure_before += __popc(stay);
    }
    if (out != nullptr)
        for (int i = a.n_keep + rank * kChooseThreads + tid; i < len; i += P * kChooseThreads) out[i] = 0.f;
    if (P > 1) cluster_sync_all();  // nobody's shared memory goes while another reads it
}

// ---------------------------------------------------------------------------------- rows
constexpr int kRowThreads = 256;
constexpr int kRowStages = 3;
constexpr int kStretchBytes = 16384;  // of a CTA

template <int P2>  // log2 of the cluster's CTAs, 0 .. 3
__global__ void __launch_bounds__(kRowThreads) evict_rows_kernel(const EvictRowsArgs a) {
    constexpr int P = 1 << P2;
    extern __shared__ __align__(128) unsigned char stages[];  // [kRowStages][kStretchBytes]
    __shared__ int src[kRowStages + 1][kStretchBytes / 128];  // a row of at least 128 bytes each; -1: none
    const int tid = threadIdx.x, rank = (int)(blockIdx.x & (P - 1));
    const int64_t unit = blockIdx.x >> P2;
    const int64_t bh = unit >> 1;
    const int b = (int)(bh / a.n_kv_heads), hk = (int)(bh % a.n_kv_heads);
    const int32_t *kept = a.kept + bh * a.n_keep;
    unsigned char *base = static_cast<unsigned char *>(unit & 1 ? a.v : a.k) + (int64_t)b * a.cache_seq + (int64_t)hk * a.cache_head;
    const int vecs = a.row_bytes / 16, rows = kStretchBytes / a.row_bytes;  // of a stretch
    const int n_stretches = (a.n_keep + P * rows - 1) / (P * rows);
    // Where row i of this CTA's stretch s comes from: threads below `rows` read the list one stretch
    // ahead of the copies.
    auto source = [&](int s) {
        const int64_t i = ((int64_t)s * P + rank) * rows + tid;
        if (tid >= rows || s >= n_stretches || i >= a.n_keep) return -1;
        const int j = __ldg(kept + i), before = i > 0 ? __ldg(kept + i - 1) : -1;
        if (j == -1) return -1;
        if (j < 0 || j >= a.capacity || j <= before || (i > 0 && before < 0)) {
            report_status(a.status, kErrBounds);
            return -1;
        }
        return j == i ? -1 : j;
    };
    auto fetch = [&](int s) {  // stretch s into its stage
        unsigned char *to = stages + s % kRowStages * kStretchBytes;
        const int *from = src[s % (kRowStages + 1)];
        if (s < n_stretches)
            for (int v = tid; v < rows * vecs; v += kRowThreads) {
                const int r = v / vecs, j = from[r];
                if (j >= 0) cp_async_16(to + v * 16, base + (int64_t)j * a.cache_rs + (v - r * vecs) * 16, true);
            }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < kRowStages; ++s)
        if (tid < rows) src[s][tid] = source(s);
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kRowStages - 1; ++s) fetch(s);
    for (int s = 0; s < n_stretches; ++s) {
        const int next = source(s + kRowStages);
        fetch(s + kRowStages - 1);
        cp_async_wait<kRowStages - 1>();  // this thread's share of stretch s
        if (tid < rows) src[(s + kRowStages) % (kRowStages + 1)][tid] = next;
        if constexpr (P > 1) cluster_sync_all();  // everyone's
        else __syncthreads();
        const unsigned char *here = stages + s % kRowStages * kStretchBytes;
        const int *from = src[s % (kRowStages + 1)];
        const int64_t i0 = ((int64_t)s * P + rank) * rows;
        for (int v = tid; v < rows * vecs; v += kRowThreads) {
            const int r = v / vecs;
            if (from[r] >= 0)
                *reinterpret_cast<uint4 *>(base + (i0 + r) * a.cache_rs + (v - r * vecs) * 16) = *reinterpret_cast<const uint4 *>(here + v * 16);
        }
        __syncthreads();  // the stage and the list's entries may be filled again
    }
    cp_async_wait<0>();
}

template <typename Kernel, typename Args>
cudaError_t launch_cluster(Kernel *k, const Args &a, int64_t grid, int threads, int smem, int cluster, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_evict_choose(EvictChooseArgs a, cudaStream_t s) {
    a.cluster = 1;
    while (a.cluster < kEvictCluster && (int64_t)a.cluster * kSliceWanted < a.max_kv_len) a.cluster *= 2;
    const int slice = (a.max_kv_len + a.cluster - 1) / a.cluster;
    static_assert(sizeof(Choose) + 4 * kEvictMaxSlice <= 232448, "shared memory budget");
    return launch_cluster(evict_choose_kernel, a, (int64_t)a.batch * a.n_kv_heads * a.cluster, kChooseThreads,
                          (int)sizeof(Choose) + 4 * slice, a.cluster, s);
}

cudaError_t launch_evict_rows(const EvictRowsArgs &a, int num_sms, cudaStream_t s) {
    const int64_t units = (int64_t)a.batch * a.n_kv_heads * 2;
    const int rows = kStretchBytes / a.row_bytes;
    // CTAs for four on every SM, as far as there are stretches for them
    int p2 = 0;
    while (p2 < 3 && (units << p2) < 4 * (int64_t)num_sms && ((int64_t)rows << p2) < a.n_keep) ++p2;
    const int smem = kRowStages * kStretchBytes;
    switch (p2) {
        case 0: return launch_cluster(evict_rows_kernel<0>, a, units, kRowThreads, smem, 1, s);
        case 1: return launch_cluster(evict_rows_kernel<1>, a, units << 1, kRowThreads, smem, 2, s);
        case 2: return launch_cluster(evict_rows_kernel<2>, a, units << 2, kRowThreads, smem, 4, s);
        default: return launch_cluster(evict_rows_kernel<3>, a, units << 3, kRowThreads, smem, 8, s);
    }
}

}  // namespace lat
