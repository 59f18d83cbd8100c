// evict.cu — the cached keys of each KV head that stay, by the attention weight they were given,
// and their rows moved up in place.
//
// choose: a cluster of up to eight CTAs takes one (sequence, KV head).  Each CTA reads its slice of
// the weights once, into shared memory (as order-preserving integers); what follows runs there.  The
// n-th largest weight is found digit by digit (11, 11 and 10 bits), counting a digit's keys into
// 2048 bins whose 16-bit counts the cluster's CTAs read from each other; it is done early where all
// keys with the prefix stay, which two digits mostly bring about.  Then a key stays if it is among
// the first or the last, is above that weight, or equals it and few equal ones come before it;
// ballots and a scan over warps and CTAs give its place, so lists are ascending, ties go to the
// lowest key, and nothing depends on an order of execution.  Since the weights wait in shared memory,
// they may be written over the ones they came from.
// What bounds it: the loops over a slice (a third of them shared atomics) and barriers and round
// trips within the cluster, then HBM (4 bytes a key).  32 heads of 65536 keys, a quarter kept: 22 us;
// clusters of 2 35, of 8 (more CTAs than SMs) 44.  Masks kept between the loops over the places
// and bins of their own for odd lanes brought nothing.
//
// rows: row i of a head becomes its row kept[i] >= i, for ascending i.  A cluster takes K or V of one
// (sequence, KV head) and moves a stretch of rows at a time: asynchronous copies bring them to shared
// memory some stretches ahead, and a stretch is written only when every CTA of the cluster says that
// its part of it has come (arrivals on barriers in each other's shared memory, which run ahead like
// the copies).  That is all the order that is needed: what a stretch writes lies before every row
// that a later one reads.  Rows that stay where they are are not touched.
// What bounds it: HBM, rows read and written once.
#include "cache_kernels.h"
#include "device_common.cuh"

namespace lat {

namespace {

// ---------------------------------------------------------------------------------- choose
constexpr int kChooseThreads = 1024, kChooseWarps = kChooseThreads / 32;
constexpr int kBins = 2048, kMyBins = kBins / kChooseThreads;
constexpr int kAtOnce = 4;  // keys of a lane at once, for the places
constexpr int kLoads = 8;   // of a thread, under way at once
// Keys of a CTA below which a larger cluster costs more talk than it saves (8 heads of 4097 keys,
// rows moved: 17.3 us, in clusters of two 18.7).
constexpr int kSliceLeast = 8192;

// order-preserving: larger weights to larger integers, NaN above all, -0 as 0
__device__ __forceinline__ uint32_t ordered(float f) {
    if (f != f) return 0xffffffffu;
    const uint32_t b = __float_as_uint(f + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float weight_of(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }
__device__ __forceinline__ uint32_t load_cluster(const void *p, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(p, rank)));
    return v;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// the sum of x over the warp's lanes before this one, and over all
__device__ __forceinline__ int warp_before(int x, int &all) {
    const int lane = threadIdx.x & 31;
    int incl = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
    }
    all = __shfl_sync(0xffffffffu, incl, 31);
    return incl - x;
}
// the sum of x over the CTA's threads before this one; `warps` in shared memory, read by all
__device__ __forceinline__ int scan_before(int x, int *warps) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int all;
    const int before = warp_before(x, all);
    if (lane == 0) warps[warp] = all;
    __syncthreads();
    return before + __reduce_add_sync(0xffffffffu, lane < warp ? warps[lane] : 0);
}

struct Choose {  // in shared memory, one a CTA
    alignas(16) uint32_t bins[kBins];
    uint32_t told[2][kBins / 2];                 // this CTA's counts for the others, two bins a word
    int warps[kChooseWarps];
    int ties[kChooseWarps], sure[kChooseWarps];  // by warp
    int all_ties, all_sure;
    uint32_t digit;
    int above, in;   // keys in the digits above, and in that one
};

template <int P>  // CTAs of a cluster
__global__ void __launch_bounds__(kChooseThreads) evict_choose_kernel(const EvictChooseArgs a) {
    extern __shared__ __align__(16) unsigned char raw[];
    Choose &sh = *reinterpret_cast<Choose *>(raw);
    uint32_t *held = reinterpret_cast<uint32_t *>(raw + sizeof(Choose));  // the slice's weights, as ordered()
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)(blockIdx.x % P);
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
        // (counted without a sign: a list may be nearly 2^31 entries long)
        for (uint32_t i = rank * kChooseThreads + tid; i < (uint32_t)a.n_keep; i += P * kChooseThreads)
            kept[i] = i < (uint32_t)len ? (int)i : -1;
        if (out != nullptr && out != w)
            for (int i = rank * kChooseThreads + tid; i < len; i += P * kChooseThreads) out[i] = w[i];
        return;
    }
    // ---- this CTA's slice, and the counts of the first digit ---------------------------------
    const int slice = (len + P - 1) / P, lo = min(len, rank * slice), n = min(len, lo + slice) - lo;
    const int mid_lo = a.n_first, mid_hi = len - a.n_last;  // keys that are chosen among
    auto chosen_among = [&](int i) { return lo + i >= mid_lo && lo + i < mid_hi; };
    uint2 *my_bins = reinterpret_cast<uint2 *>(sh.bins) + (kChooseThreads - 1 - tid);  // thread 0: the largest digits
    *my_bins = make_uint2(0, 0);
    __syncthreads();
    for (int i0 = tid; i0 < n; i0 += kLoads * kChooseThreads) {
        float v[kLoads];
#pragma unroll
        for (int q = 0; q < kLoads; ++q) {
            const int i = i0 + q * kChooseThreads;
            v[q] = i < n ? __ldcg(w + lo + i) : 0.f;  // (they may be written over)
        }
#pragma unroll
        for (int q = 0; q < kLoads; ++q) {
            const int i = i0 + q * kChooseThreads;
            if (i >= n) continue;
            const uint32_t k = ordered(v[q]);
            held[i] = k;
            if (chosen_among(i)) atomicAdd(&sh.bins[k >> 21], 1u);
        }
    }

    // ---- the weight that the last chosen key has, digit by digit ---------------------------------
    int need = a.n_keep - a.n_first - a.n_last;  // keys still to be chosen among those with the prefix
    uint32_t prefix = 0, mask = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3 && need > 0; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        if (pass > 0) {
#pragma unroll 4
            for (int i = tid; i < n; i += kChooseThreads) {
                const uint32_t k = held[i];
                if ((k & mask) == prefix && chosen_among(i)) atomicAdd(&sh.bins[(k >> shift) & ((1u << bits) - 1)], 1u);
            }
        }
        __syncthreads();
        // the cluster's counts, largest digits first: thread t has two, and what lies above
        const uint2 mine = *my_bins;
        *my_bins = make_uint2(0, 0);
        uint32_t c[kMyBins] = {mine.y, mine.x};
        if constexpr (P > 1) {
            // (a slice's counts fit 16 bits; the words of the last pass but one have been read by all)
            sh.told[pass & 1][tid] = mine.y | mine.x << 16;
            cluster_sync_all();
            uint32_t part[P];
#pragma unroll
            for (int p = 1; p < P; ++p) part[p] = load_cluster(&sh.told[pass & 1][tid], (uint32_t)((rank + p) % P));
#pragma unroll
            for (int p = 1; p < P; ++p) c[0] += part[p] & 0xffffu, c[1] += part[p] >> 16;
        }
        int above = scan_before((int)(c[0] + c[1]), sh.warps);
#pragma unroll
        for (int q = 0; q < kMyBins; ++q) {
            if (above < need && above + (int)c[q] >= need)
                sh.digit = kBins - 1 - (kMyBins * tid + q), sh.above = above, sh.in = (int)c[q];
            above += (int)c[q];
        }
        __syncthreads();
        prefix |= sh.digit << shift;
        mask |= ((1u << bits) - 1) << shift;
        need -= sh.above;
        if (need == sh.in) break;  // all keys with this prefix stay: no further digit tells them apart
    }
    // ---- places: a warp takes a run of the slice, in order ------------------------------------------
    // a key's rank: 2 stays, 1 is one of the equal ones, 0 goes
    constexpr int kStep = 32 * kAtOnce;
    const bool none = a.n_keep == a.n_first + a.n_last;
    auto ranks = [&](int i0, uint32_t (&k)[kAtOnce], int (&r)[kAtOnce]) {
        if (i0 + kStep <= n && lo + i0 >= mid_lo && lo + i0 + kStep <= mid_hi && !none) {
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) k[q] = held[i0 + 32 * q + lane];
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) r[q] = (k[q] & mask) > prefix ? 2 : (k[q] & mask) == prefix ? 1 : 0;
            return;
        }
#pragma unroll 1
        for (int q = 0; q < kAtOnce; ++q) {
            const int i = i0 + 32 * q + lane;
            const uint32_t x = i < n ? held[i] : 0, m = x & mask;
            const int at = i >= n ? 0 : !chosen_among(i) ? 2 : none ? 0 : m > prefix ? 2 : m == prefix ? 1 : 0;
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u)
                if (u == q) k[u] = x, r[u] = at;
        }
    };
    const int run = (slice + kChooseWarps * kStep - 1) / (kChooseWarps * kStep) * kStep;  // keys of a warp
    const int run_end = min((warp + 1) * run, n);
    int ties = 0, sure = 0;
    for (int i0 = warp * run; i0 < run_end; i0 += kStep) {
        uint32_t k[kAtOnce];
        int r[kAtOnce];
        ranks(i0, k, r);
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) ties += r[q] == 1, sure += r[q] == 2;
    }
    ties = __reduce_add_sync(0xffffffffu, ties), sure = __reduce_add_sync(0xffffffffu, sure);
    if (lane == 0) sh.ties[warp] = ties, sh.sure[warp] = sure;
    __syncthreads();
    int all_ties, all_sure;  // of the CTA
    const int ties_ahead = warp_before(sh.ties[lane], all_ties), sure_ahead = warp_before(sh.sure[lane], all_sure);
    int ties_before = __shfl_sync(0xffffffffu, ties_ahead, warp), sure_before = __shfl_sync(0xffffffffu, sure_ahead, warp);
    if constexpr (P > 1) {
        if (tid == 0) sh.all_ties = all_ties, sh.all_sure = all_sure;
        cluster_sync_all();
        const bool earlier = lane < rank;  // (a CTA a lane)
        ties_before += __reduce_add_sync(0xffffffffu, earlier ? (int)load_cluster(&sh.all_ties, (uint32_t)lane) : 0);
        sure_before += __reduce_add_sync(0xffffffffu, earlier ? (int)load_cluster(&sh.all_sure, (uint32_t)lane) : 0);
        cluster_arrive();  // (the others' shared memory has been read)
    }
    const uint32_t under = (1u << lane) - 1;
    for (int i0 = warp * run; i0 < run_end; i0 += kStep) {
        uint32_t k[kAtOnce];
        int r[kAtOnce];
        ranks(i0, k, r);
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) {
            const uint32_t tied = __ballot_sync(0xffffffffu, r[q] == 1), stay = __ballot_sync(0xffffffffu, r[q] == 2);
            // sure ones before, and the equal ones before that stay
            int at = sure_before + __popc(stay & under) + min(ties_before, need);
            bool stays = r[q] == 2;
            if (tied != 0) {
                const int t = ties_before + __popc(tied & under);
                at += min(t, need) - min(ties_before, need);
                stays |= r[q] == 1 && t < need;
                ties_before += __popc(tied);
            }
            if (stays) {
                kept[at] = lo + i0 + 32 * q + lane;
                if (out != nullptr) out[at] = weight_of(k[q]);
            }
            sure_before += __popc(stay);
        }
    }
    if (out != nullptr)
        for (int i = a.n_keep + rank * kChooseThreads + tid; i < len; i += P * kChooseThreads) out[i] = 0.f;
    if (P > 1) cluster_wait();  // nobody's shared memory goes while another reads it
}

// ---------------------------------------------------------------------------------- rows
constexpr int kRowThreads = 256;
constexpr int kRowStages = 3;
constexpr int kStretchBytes = 32768;  // of a CTA
constexpr int kPieces = kStretchBytes / 16 / kRowThreads;  // 16-byte pieces of a thread
constexpr int kRowBars = 2 * kRowStages;

template <int P2>  // log2 of the cluster's CTAs, 0 .. 3
__global__ void __launch_bounds__(kRowThreads) evict_rows_kernel(const EvictRowsArgs a) {
    constexpr int P = 1 << P2;
    extern __shared__ __align__(128) unsigned char stages[];  // [kRowStages][kStretchBytes]
    __shared__ int src[kRowStages + 1][kStretchBytes / 128];  // rows of at least 128 bytes; -1: none
    // Stretch s has come to all CTAs.  A CTA that says so of stretch s + kRowBars has seen this one say
    // it of s + kRowStages, and so be done with s: twice as many barriers as stages, each a phase at
    // a time.
    __shared__ __align__(8) uint64_t here[kRowBars];
    __shared__ int abort_flag;
    const int tid = threadIdx.x, rank = (int)(blockIdx.x & (P - 1));
    const int64_t unit = blockIdx.x >> P2;
    const int64_t bh = unit >> 1;
    const int b = (int)(bh / a.n_kv_heads), hk = (int)(bh % a.n_kv_heads);
    const int32_t *kept = a.kept + bh * a.n_keep;
    unsigned char *base = static_cast<unsigned char *>(unit & 1 ? a.v : a.k) + (int64_t)b * a.cache_seq + (int64_t)hk * a.cache_head;
    const int vecs = a.row_bytes / 16, rows = kStretchBytes / a.row_bytes;  // of a stretch
    // (no entry from the capacity on can be a row: ascending, it would be past it)
    const int n_rows = min(a.n_keep, a.capacity), n_stretches = (int)(((int64_t)n_rows + P * rows - 1) / (P * rows));
    const uint64_t deadline = globaltimer_ns() + a.timeout_ns;
    // this thread's pieces of a stretch: row and byte within it
    int row[kPieces], off[kPieces];
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
        const int v = tid + k * kRowThreads;
        row[k] = v / vecs;
        off[k] = (v - row[k] * vecs) * 16;
        if (row[k] >= rows) row[k] = -1;
    }
    // Where row i of this CTA's stretch s comes from: threads below `rows` read the list one stretch
    // ahead of the copies.
    auto source = [&](int s) {
        const int64_t i = ((int64_t)s * P + rank) * rows + tid;
        if (tid >= rows || s >= n_stretches || i >= n_rows) return -1;
        const int j = __ldg(kept + i), before = i > 0 ? __ldg(kept + i - 1) : -1;
        if (j == -1) return -1;
        if (j < i || j >= a.capacity || j <= before || (i > 0 && before < 0)) {  // (ascending lists never have j < i)
            report_status(a.status, kErrBounds);
            return -1;
        }
        return j == i ? -1 : j;
    };
    auto fetch = [&](int s) {  // stretch s into its stage
        unsigned char *to = stages + s % kRowStages * kStretchBytes;
        const int *from = src[s % (kRowStages + 1)];
        if (s < n_stretches)
#pragma unroll
            for (int k = 0; k < kPieces; ++k) {
                const int j = row[k] >= 0 ? from[row[k]] : -1;
                if (j >= 0) cp_async_16(to + (tid + k * kRowThreads) * 16, base + (int64_t)j * a.cache_rs + off[k], true);
            }
        cp_async_commit();
    };
    auto tell = [&](int s) {  // (behind a barrier of this CTA's threads)
        if constexpr (P > 1)
            if (tid < P && s < n_stretches && !(a.test_skip_tell && rank + s == 0)) mbar_arrive_cluster(cluster_addr(&here[s % kRowBars], (uint32_t)tid));
    };
    if (!(unit & 1) && a.n_keep > n_rows) {  // what is not read below has to be -1
        bool none = true;
        for (uint32_t i = (uint32_t)n_rows + rank * kRowThreads + tid; i < (uint32_t)a.n_keep; i += P * kRowThreads)
            none &= __ldg(kept + i) == -1;
        if (!none) report_status(a.status, kErrBounds);
    }
    if (tid == 0) {
        for (int i = 0; i < kRowBars; ++i) mbar_init(&here[i], P);
        fence_mbarrier_init();
        abort_flag = 0;
    }
#pragma unroll
    for (int s = 0; s < kRowStages; ++s)
        if (tid < rows) src[s][tid] = source(s);
    if constexpr (P > 1) cluster_sync_all();  // everyone's barriers are there
    else __syncthreads();
#pragma unroll
    for (int s = 0; s < kRowStages - 1; ++s) fetch(s);
    cp_async_wait<kRowStages - 2>();
    __syncthreads();
    tell(0);
    for (int s = 0; s < n_stretches; ++s) {
        const int next = source(s + kRowStages);
        fetch(s + kRowStages - 1);
        cp_async_wait<kRowStages - 2>();  // this thread's pieces of stretch s + 1
        if (tid < rows) src[(s + kRowStages) % (kRowStages + 1)][tid] = next;
        if (P > 1 && tid == 0) mbar_wait_bounded_cluster(&here[s % kRowBars], (s / kRowBars) & 1, &abort_flag, deadline);
        __syncthreads();
        if (P > 1 && abort_flag) break;  // (one thread's word, seen by all alike)
        tell(s + 1);
        const unsigned char *from_stage = stages + s % kRowStages * kStretchBytes;
        const int *from = src[s % (kRowStages + 1)];
        const int64_t i0 = ((int64_t)s * P + rank) * rows;
#pragma unroll
        for (int k = 0; k < kPieces; ++k)
            if (row[k] >= 0 && from[row[k]] >= 0)
                *reinterpret_cast<uint4 *>(base + (i0 + row[k]) * a.cache_rs + off[k]) =
                    *reinterpret_cast<const uint4 *>(from_stage + (tid + k * kRowThreads) * 16);
        __syncthreads();  // the stage and the list's entries may be filled again
    }
    cp_async_wait<0>();
    if constexpr (P > 1) {
        __syncthreads();
        if (tid == 0 && abort_flag) report_status(a.status, kErrTimeout);
        cluster_sync_all();  // nobody's barriers go while another arrives on them
    }
}

// `most`: the most shared memory that the kernel is ever given
template <typename Kernel, typename Args>
cudaError_t launch_cluster(Kernel *k, SharedLimit &limit, int most, const Args &a, int64_t grid, int threads, int smem,
                           int cluster, cudaStream_t s) {
    cudaError_t e = limit(k, most);
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

cudaError_t launch_evict_choose(EvictChooseArgs a, int num_sms, cudaStream_t s) {
    a.cluster = 1;
    // more CTAs a head while its slices do not fit, or while there are SMs for them (256 heads of 32768
    // keys, rows moved: 98 us, in clusters of two 102)
    const int64_t units = (int64_t)a.batch * a.n_kv_heads;
    while (a.cluster < kEvictCluster && ((int64_t)a.cluster * kEvictMaxSlice < a.max_kv_len ||
                                         (units * a.cluster * 2 <= num_sms && a.cluster * kSliceLeast < a.max_kv_len)))
        a.cluster *= 2;
    const int slice = (a.max_kv_len + a.cluster - 1) / a.cluster;
    static_assert(kMyBins == 2 && kChooseWarps == 32, "pairs of bins, a warp a lane");
    static_assert(sizeof(Choose) + 4 * kEvictMaxSlice <= 232448, "shared memory budget");
    const int64_t grid = (int64_t)a.batch * a.n_kv_heads * a.cluster;
    const int most = (int)sizeof(Choose) + 4 * kEvictMaxSlice, smem = (int)sizeof(Choose) + 4 * slice;
    static SharedLimit limit[4];
    switch (a.cluster) {
        case 1: return launch_cluster(evict_choose_kernel<1>, limit[0], most, a, grid, kChooseThreads, smem, 1, s);
        case 2: return launch_cluster(evict_choose_kernel<2>, limit[1], most, a, grid, kChooseThreads, smem, 2, s);
        case 4: return launch_cluster(evict_choose_kernel<4>, limit[2], most, a, grid, kChooseThreads, smem, 4, s);
        default: return launch_cluster(evict_choose_kernel<8>, limit[3], most, a, grid, kChooseThreads, smem, 8, s);
    }
}

cudaError_t launch_evict_rows(const EvictRowsArgs &a, int num_sms, cudaStream_t s) {
    const int64_t units = (int64_t)a.batch * a.n_kv_heads * 2;
    const int rows = kStretchBytes / a.row_bytes;
    // CTAs for two on every SM, as many as fit there at once, as far as there are stretches for them
    int p2 = 0;
    while (p2 < 3 && (units << (p2 + 1)) <= 2 * (int64_t)num_sms && ((int64_t)rows << p2) < a.n_keep) ++p2;
    const int smem = kRowStages * kStretchBytes;
    static SharedLimit limit[4];
    switch (p2) {
        case 0: return launch_cluster(evict_rows_kernel<0>, limit[0], smem, a, units, kRowThreads, smem, 1, s);
        case 1: return launch_cluster(evict_rows_kernel<1>, limit[1], smem, a, units << 1, kRowThreads, smem, 2, s);
        case 2: return launch_cluster(evict_rows_kernel<2>, limit[2], smem, a, units << 2, kRowThreads, smem, 4, s);
        default: return launch_cluster(evict_rows_kernel<3>, limit[3], smem, a, units << 3, kRowThreads, smem, 8, s);
    }
}

}  // namespace lat
