// decode_q4.cu — split-KV decode over a 4-bit KV cache (the row format: q4_row.cuh).
//
// What it computes: for each sequence b and query head h, attention of one query row over
// the visible cached keys, with key and value channel d of group g read as s_jg (c_jd - z_jg):
//   x_j = scale * sum_g s_jg sum_{d in g} q_d (c_jd - z_jg)      (then capped, if asked for)
//   out = sum_j e^{x_j - m} v_j / sum_j e^{x_j - m}
// The scale never meets the codes: a group's products are summed by the tensor cores and
// scaled once per key, and V's scales multiply the softmax weights, p_j s_jg, before their
// one rounding to bf16.
//
// How:
//  * Work unit = one (sequence, KV head, block of <= 8 query heads).  All units' keys, laid
//    end to end in tiles of kTileKeys, form one stream; CTA c takes the c-th equal share
//    (never under min_tiles).  A unit cut across CTAs leaves one normalised partial and its
//    log-sum-exp per piece, joined by a second kernel (a programmatic dependent).
//  * Every warp is its own pipeline: it owns kKeys rows of each tile, which one TMA copy
//    brings into its ring (a box over the cache's strides; the row is one run of bytes for
//    K and V), and its first lane issues the copy for a stage as soon as the warp is done
//    with it.  Warps meet only at the end of a piece.
//  * mma m16n8k16 with keys in M: S^T[16 keys x 8 heads] = K Q^T by groups of 32 channels,
//    O^T[16 channels x 8 heads] += V^T (P s)^T.  A word of codes becomes four bf16 pairs of
//    128 + c by an AND-OR each (0x4300 is bf16 128, whose last place is 1), minus 128 + z,
//    which is exact.  The rows' layout puts a lane's codes side by side.
//  * LAT_F32: the query, and the weights p s, are split into three bf16 terms (24 bits, so
//    nothing is lost); the codes are exact as they are, so three MMAs give fp32 products.
//  * Waits are bounded; on expiry the CTA records LAT_ERR_TIMEOUT, drains its copies, quits.
#include <math.h>

#include <algorithm>

#include "device_common.cuh"
#include "kernels.h"
#include "q4_row.cuh"
#include "split_join.cuh"

namespace lat {

namespace {

constexpr int kHeads = 8;                  // N of the mma: query heads of a unit
constexpr float kRescaleBy = 8.0f;         // log2 units the maximum may grow unnoticed
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kPieceRing = 8;              // pieces known ahead

template <int D, bool F32>
struct Q4Cfg {
    using R = Q4Row<D>;
    static constexpr int kWarps = 4;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kTerms = F32 ? 3 : 1;               // bf16 terms of q and of p s
    static constexpr int kSub = D == 512 ? 1 : 2;            // 16-key MMA tiles a warp takes at once
    static constexpr int kKeys = 16 * kSub;
    static constexpr int kTileKeys = kKeys * kWarps;
    static constexpr int kStages = 3;
    static constexpr int kStageBytes = kKeys * R::kBytes;
    static constexpr int kMt = D / 16;                       // 16-channel MMA tiles
    static constexpr bool kQReg = R::kPad * kTerms <= 256;   // query fragments in registers
    static constexpr int kQPitch = R::kPad + 32;             // bf16; rows 16 words apart in the banks
    static constexpr int kQBytes = kQReg ? 0 : kTerms * kHeads * kQPitch * 2;
    static constexpr int kRound = 4;                         // MMA tiles joined at once: 64 channels
    static constexpr int kParkPitch = 16 * kRound + 4;
    static constexpr int kParkBytes = kWarps * kHeads * kParkPitch * 4;
    static constexpr int kMisc = 1024;
    static constexpr int kSmem = kWarps * kStages * kStageBytes + kQBytes + kParkBytes + kMisc;
    static_assert(kSmem <= 232448, "shared memory budget");
    static_assert(kStageBytes % 128 == 0, "TMA destinations");
};

struct Piece {
    int b, hk, hb;     // unit
    int key0, keys;    // first key, keys of the piece (the last tile may be partial)
    int slot, nseg;    // which piece of how many
    int end;           // no more pieces
};

struct KeyRange {
    int lo, n;
};
__device__ __forceinline__ KeyRange range_of(const Q4DecodeArgs &a, int len) {
    KeyRange k{0, 0};
    if (len < 0 || len > a.max_kv_len) return k;  // reported once, by CTA 0
    k.lo = a.window > 0 ? max(0, len - a.window) : 0;
    k.n = len - k.lo;
    return k;
}

// thread 0's place in the stream
struct Walk {
    long long pos, end, pb, per_cta;  // pb: where sequence b's units begin
    int b;
};

template <int T>
__device__ bool next_piece(const Q4DecodeArgs &a, Walk &w, int HB, Piece &p) {
    const int HU = a.n_kv_heads * HB;
    while (w.pos < w.end && w.b < a.batch) {
        const KeyRange k = range_of(a, a.kv_lens[w.b]);
        const int nt = (k.n + T - 1) / T;
        const long long all = (long long)nt * HU;
        if (w.pos >= w.pb + all) {
            w.pb += all;
            ++w.b;
            continue;
        }
        const int idx = (int)((w.pos - w.pb) / nt);
        const long long ustart = w.pb + (long long)idx * nt;
        const int t0 = (int)(w.pos - ustart), t1 = (int)min((long long)nt, w.end - ustart);
        const long long first = ustart / w.per_cta, last = (ustart + nt - 1) / w.per_cta;
        p.b = w.b;
        p.hk = idx / HB;
        p.hb = idx % HB;
        p.key0 = k.lo + t0 * T;
        p.keys = min(k.n, t1 * T) - t0 * T;
        p.slot = (int)(blockIdx.x - first);
        p.nseg = (int)(last - first + 1);
        p.end = 0;
        w.pos = ustart + t1;
        return true;
    }
    p.end = 1;
    return false;
}

// N consecutive 32-bit words of shared memory, in the widest loads their count allows
template <int N>
__device__ __forceinline__ void lds_words(uint32_t (&w)[N], const unsigned char *p) {
    if constexpr (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x, w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = reinterpret_cast<const uint32_t *>(p)[i];
    }
}
// a lane's V halves of one set from two rows, paired: low halves from row x, high from row y
template <int SET>
__device__ __forceinline__ void v_pairs(uint32_t (&u)[SET], const unsigned char *x, const unsigned char *y) {
    if constexpr (SET % 2 == 0) {
        uint32_t wx[SET / 2], wy[SET / 2];
        if constexpr (SET == 4) {
            lds_words(wx, x);
            lds_words(wy, y);
        } else {
            wx[0] = *reinterpret_cast<const uint32_t *>(x);
            wy[0] = *reinterpret_cast<const uint32_t *>(y);
        }
#pragma unroll
        for (int j = 0; j < SET; ++j) u[j] = __byte_perm(wx[j / 2], wy[j / 2], (j & 1) ? 0x7632 : 0x5410);
    } else {
#pragma unroll
        for (int j = 0; j < SET; ++j)
            u[j] = (uint32_t)reinterpret_cast<const uint16_t *>(x)[j] |
                   ((uint32_t)reinterpret_cast<const uint16_t *>(y)[j] << 16);
    }
}

// two floats as `TERMS` packed bf16 pairs whose sum is the pair (to 8 bits a term)
template <int TERMS>
__device__ __forceinline__ void split2(uint32_t (&o)[TERMS], float x, float y) {
#pragma unroll
    for (int t = 0; t < TERMS; ++t) {
        o[t] = pack_bf16x2(x, y);
        if (t + 1 < TERMS) {
            x -= __uint_as_float(o[t] << 16);
            y -= __uint_as_float(o[t] & 0xffff0000u);
        }
    }
}

template <int D, bool F32>
__global__ void __launch_bounds__(Q4Cfg<D, F32>::kThreads)
decode_q4_kernel(const __grid_constant__ Q4DecodeArgs a) {
    using C = Q4Cfg<D, F32>;
    using R = Q4Row<D>;
    using T = typename std::conditional<F32, float, __nv_bfloat16>::type;
    constexpr int kTerms = C::kTerms, kSet = R::kSet, kSets = R::kGroups / R::kSet;
    extern __shared__ __align__(128) unsigned char smem[];  // (an aligned-up pointer would load as generic)
    unsigned char *ring = smem;                                              // [warp][stage]
    unsigned char *sQ = ring + C::kWarps * C::kStages * C::kStageBytes;      // [term][head] rows
    float *park = reinterpret_cast<float *>(sQ + C::kQBytes);                // [warp][head][channel]
    unsigned char *misc = reinterpret_cast<unsigned char *>(park) + C::kParkBytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(misc);                     // [warp][stage]
    Piece *pieces = reinterpret_cast<Piece *>(misc + 128);                   // [kPieceRing]
    float *sM = reinterpret_cast<float *>(misc + 384);                       // [warp][m[8], l[8]]
    Walk *walk = reinterpret_cast<Walk *>(misc + 640);
    long long *scan = reinterpret_cast<long long *>(misc + 704);             // [warps]
    volatile int *abort_flag = reinterpret_cast<int *>(misc + 768);
    static_assert(sizeof(Piece) * kPieceRing <= 256 && sizeof(Walk) <= 64, "misc area");

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.n_heads / a.n_kv_heads, HB = (G + kHeads - 1) / kHeads, HU = a.n_kv_heads * HB;
    constexpr int TK = C::kTileKeys;

    // ---- the stream's length and this CTA's share: per-thread sums over a slice of the
    // sequences, then a scan ------------------------------------------------------------
    const int per_thread = (a.batch + C::kThreads - 1) / C::kThreads;
    const int b_lo = min(a.batch, tid * per_thread), b_hi = min(a.batch, b_lo + per_thread);
    long long my_sum = 0;
    for (int b = b_lo; b < b_hi; ++b) {
        const int len = a.kv_lens[b];
        const KeyRange k = range_of(a, len);
        my_sum += (long long)((k.n + TK - 1) / TK) * HU;
        if (blockIdx.x == 0 && k.n == 0) {  // nothing to stream
            const bool bad = len < 0 || len > a.max_kv_len;
            if (bad) report_status(a.status, kErrBounds);
            for (int h = 0; h < a.n_heads; ++h) {
                a.piece_count[(int64_t)b * a.n_heads + h] = 0;
                if (!bad && a.lse != nullptr) a.lse[(int64_t)b * a.n_heads + h] = -INFINITY;
            }
            if (!bad)
                for (int i = 0; i < a.n_heads * D; ++i) static_cast<T *>(a.out)[(int64_t)b * a.out_rs + i] = T(0.f);
        }
    }
    long long incl = my_sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
    }
    if (lane == 31) scan[warp] = incl;
    if (tid == 0) {
        walk->pos = 0;
        walk->end = 0;
        walk->b = a.batch;
        for (int i = 0; i < C::kWarps * C::kStages; ++i) mbar_init(&full[i], 1);
        *abort_flag = 0;
        fence_mbarrier_init();
    }
    __syncthreads();
    long long total = 0, my_start = incl - my_sum;
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w) {
        const long long v = scan[w];
        if (w < warp) my_start += v;
        total += v;
    }
    const long long per_cta = max((total + gridDim.x - 1) / gridDim.x, (long long)a.min_tiles);
    const long long r0 = (long long)blockIdx.x * per_cta, r1 = min(total, r0 + per_cta);
    if (r0 < r1 && r0 >= my_start && r0 < my_start + my_sum) {  // the share begins in this slice
        long long p = my_start;
        int b = b_lo;
        for (; b < b_hi; ++b) {
            const long long w = (long long)((range_of(a, a.kv_lens[b]).n + TK - 1) / TK) * HU;
            if (r0 < p + w) break;
            p += w;
        }
        walk->pos = r0;
        walk->end = r1;
        walk->pb = p;
        walk->b = b;
        walk->per_cta = per_cta;
    }
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (r0 >= r1) return;
    if (tid == 0) {
        Walk w = *walk;
        for (int i = 0; i < kPieceRing / 2; ++i)
            if (!next_piece<TK>(a, w, HB, pieces[i])) break;
        *walk = w;
        tma_prefetch_desc(&a.tm);
    }
    __syncthreads();
    const uint64_t deadline = globaltimer_ns() + a.timeout_ns;

    // ---- this warp's copies -------------------------------------------------------------
    unsigned char *my_ring = ring + warp * C::kStages * C::kStageBytes;
    uint64_t *my_full = full + warp * C::kStages;
    int ip = 0, it = 0;            // next copy: piece, tile of the piece
    unsigned issued = 0, used = 0; // copies issued, consumed
    // Issues this warp's next copy, if one is known.  A piece whose last tile leaves this warp
    // no row has no copy for that tile.  `limit`: pieces in the table.
    auto issue = [&](int limit) {
        while (ip < limit) {
            const Piece &p = pieces[ip % kPieceRing];
            if (p.end) return;
            const int k0 = it * TK + warp * C::kKeys;
            if (k0 >= p.keys) {  // (also where the piece is over)
                if ((it + 1) * TK >= p.keys) ++ip, it = 0;
                else ++it;
                continue;
            }
            const unsigned s = issued % C::kStages;
            if (lane == 0) {
                mbar_arrive_expect_tx(&my_full[s], C::kStageBytes);
                tma_load_4d(my_ring + s * C::kStageBytes, &a.tm, &my_full[s], 0, p.hk, p.key0 + k0, p.b);
            }
            ++issued;
            if ((it + 1) * TK >= p.keys) ++ip, it = 0;
            else ++it;
            return;
        }
    };
    int known = kPieceRing / 2;  // table entries written (or behind an end mark)
    for (int s = 0; s < C::kStages; ++s) issue(known);

    const int r = lane >> 2, c = lane & 3;
    // MMA row r is the tile's key perm(r): the two low bits swapped, so that the eight lanes of
    // a 16-byte shared-memory access fall into different banks at a 160-byte row
    const int kr = (r & 4) | ((r & 1) << 1) | ((r >> 1) & 1);
    const int kp = ((c & 2) << 1) | (c & 1);  // perm(2 c); perm(2 c + 1) is kp + 2

    for (int pi = 0;; ++pi) {
        const Piece p = pieces[pi % kPieceRing];
        if (p.end) break;
        const int h_base = p.hk * G + p.hb * kHeads, g_cnt = min(kHeads, G - p.hb * kHeads);
        // ---- the unit's queries: lane (r, c) holds head r's channels 32 g + 8 c .. + 7 -----
        uint32_t qf[C::kQReg ? R::kGroups : 1][kTerms][4];
        {
            const T *qrow = static_cast<const T *>(a.q) + (int64_t)p.b * a.q_rs + (int64_t)h_base * D;
            auto octet = [&](int head, int d, uint32_t (&o)[kTerms][4]) {  // 8 channels, in terms
                const bool live = head < g_cnt && d < D;
                if constexpr (F32) {
                    const float4 *src = reinterpret_cast<const float4 *>(qrow + (int64_t)head * D + d);
                    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
                    const float4 x = live ? src[0] : z, y = live ? src[1] : z;
                    uint32_t t[kTerms];
                    split2<kTerms>(t, x.x, x.y);
#pragma unroll
                    for (int k = 0; k < kTerms; ++k) o[k][0] = t[k];
                    split2<kTerms>(t, x.z, x.w);
#pragma unroll
                    for (int k = 0; k < kTerms; ++k) o[k][1] = t[k];
                    split2<kTerms>(t, y.x, y.y);
#pragma unroll
                    for (int k = 0; k < kTerms; ++k) o[k][2] = t[k];
                    split2<kTerms>(t, y.z, y.w);
#pragma unroll
                    for (int k = 0; k < kTerms; ++k) o[k][3] = t[k];
                } else {
                    const uint4 x = live ? *reinterpret_cast<const uint4 *>(qrow + (int64_t)head * D + d)
                                         : make_uint4(0, 0, 0, 0);
                    o[0][0] = x.x, o[0][1] = x.y, o[0][2] = x.z, o[0][3] = x.w;
                }
            };
            if constexpr (C::kQReg) {
#pragma unroll
                for (int g = 0; g < R::kGroups; ++g) octet(r, 32 * g + 8 * c, qf[g]);
            } else {
                for (int i = tid; i < kHeads * R::kPad / 8; i += C::kThreads) {
                    const int head = i / (R::kPad / 8), d = 8 * (i % (R::kPad / 8));
                    uint32_t o[kTerms][4];
                    octet(head, d, o);
#pragma unroll
                    for (int k = 0; k < kTerms; ++k)
                        *reinterpret_cast<uint4 *>(sQ + ((k * kHeads + head) * C::kQPitch + d) * 2) =
                            make_uint4(o[k][0], o[k][1], o[k][2], o[k][3]);
                }
                __syncthreads();
            }
        }
        float m_ref[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
        float acc[C::kMt][4];
#pragma unroll
        for (int i = 0; i < C::kMt; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;

        for (int k0 = warp * C::kKeys; k0 < p.keys; k0 += TK) {
            const unsigned s = used % C::kStages;
            const bool got = mbar_wait_bounded(&my_full[s], (used / C::kStages) & 1, abort_flag, deadline);
            if (!__all_sync(0xffffffffu, got)) break;
            unsigned char *tile = my_ring + s * C::kStageBytes;
            const int valid = min(C::kKeys, p.keys - k0);
            if (valid < C::kKeys) {
                // rows past the end hold anything: their parameters become zeros, so that what
                // they add is a finite number times a weight of zero
                for (int i = lane; i < (C::kKeys - valid) * 2 * R::kGroups; i += 32)
                    reinterpret_cast<uint32_t *>(tile + (valid + i / (2 * R::kGroups)) * R::kBytes +
                                                 R::kParamK)[i % (2 * R::kGroups)] = 0u;
                __syncwarp();
            }
            // ---- S^T: by groups, each scaled by its keys' scales -----------------------------
            float sc[C::kSub][4];
#pragma unroll
            for (int u = 0; u < C::kSub; ++u) sc[u][0] = sc[u][1] = sc[u][2] = sc[u][3] = 0.f;
#pragma unroll
            for (int st = 0; st < kSets; ++st) {
                uint32_t qs[C::kQReg ? 1 : kSet][kTerms][4];
                if constexpr (!C::kQReg) {
#pragma unroll
                    for (int j = 0; j < kSet; ++j)
#pragma unroll
                        for (int k = 0; k < kTerms; ++k) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(
                                sQ + ((k * kHeads + r) * C::kQPitch + 32 * (st * kSet + j) + 8 * c) * 2);
                            qs[j][k][0] = v.x, qs[j][k][1] = v.y, qs[j][k][2] = v.z, qs[j][k][3] = v.w;
                        }
                }
#pragma unroll
                for (int u = 0; u < C::kSub; ++u) {
                    const unsigned char *x = tile + (16 * u + kr) * R::kBytes, *y = x + 8 * R::kBytes;
                    uint32_t wx[kSet], wy[kSet], px[kSet], py[kSet];
                    lds_words(wx, x + 4 * kSet * (4 * st + c));
                    lds_words(wy, y + 4 * kSet * (4 * st + c));
                    lds_words(px, x + R::kParamK + 4 * kSet * st);
                    lds_words(py, y + R::kParamK + 4 * kSet * st);
#pragma unroll
                    for (int j = 0; j < kSet; ++j) {
                        const uint32_t bx = q4_bias2(px[j]), by = q4_bias2(py[j]);
                        float d[4] = {0.f, 0.f, 0.f, 0.f};
                        const uint32_t a0[4] = {q4_codes2(wx[j], 0, bx), q4_codes2(wy[j], 0, by), q4_codes2(wx[j], 1, bx),
                                                q4_codes2(wy[j], 1, by)};
                        const uint32_t a1[4] = {q4_codes2(wx[j], 2, bx), q4_codes2(wy[j], 2, by), q4_codes2(wx[j], 3, bx),
                                                q4_codes2(wy[j], 3, by)};
#pragma unroll
                        for (int k = kTerms - 1; k >= 0; --k) {
                            const uint32_t(&q)[4] = [&]() -> const uint32_t(&)[4] {
                                if constexpr (C::kQReg) return qf[st * kSet + j][k];
                                else return qs[j][k];
                            }();
                            mma_bf16_16816(d, a0, q[0], q[1]);
                            mma_bf16_16816(d, a1, q[2], q[3]);
                        }
                        const float fx = q4_scale(px[j]), fy = q4_scale(py[j]);
                        sc[u][0] = fmaf(fx, d[0], sc[u][0]);
                        sc[u][1] = fmaf(fx, d[1], sc[u][1]);
                        sc[u][2] = fmaf(fy, d[2], sc[u][2]);
                        sc[u][3] = fmaf(fy, d[3], sc[u][3]);
                    }
                }
            }
            // ---- the log2 domain, the cap, the mask ------------------------------------------
            if (a.cap_log2 > 0.f) {
                const float k2 = a.raw_over_cap * kTwoLog2e;
#pragma unroll
                for (int u = 0; u < C::kSub; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sc[u][e] = F32 ? a.cap_log2 * tanhf(sc[u][e] * a.raw_over_cap)
                                       : capped_score_log2(sc[u][e], k2, a.cap_log2);
            } else {
#pragma unroll
                for (int u = 0; u < C::kSub; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[u][e] *= a.scale_log2;
            }
            if (valid < C::kKeys) {
#pragma unroll
                for (int u = 0; u < C::kSub; ++u) {
                    if (16 * u + kr >= valid) sc[u][0] = sc[u][1] = -INFINITY;
                    if (16 * u + 8 + kr >= valid) sc[u][2] = sc[u][3] = -INFINITY;
                }
            }
            // ---- running maximum and sum ----------------------------------------------------
            float corr[2];
            bool refresh_any = false;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float t = fmaxf(sc[0][e], sc[0][e + 2]);
#pragma unroll
                for (int u = 1; u < C::kSub; ++u) t = fmaxf(t, fmaxf(sc[u][e], sc[u][e + 2]));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
                const bool refresh = t > m_ref[e] + kRescaleBy;
                const float m_new = refresh ? t : m_ref[e];
                const float m_use = m_new == -INFINITY ? 0.f : m_new;
                corr[e] = refresh ? fast_exp2(m_ref[e] - m_use) : 1.f;
                float sum = 0.f;
#pragma unroll
                for (int u = 0; u < C::kSub; ++u) {
                    sc[u][e] = fast_exp2(sc[u][e] - m_use);
                    sc[u][e + 2] = fast_exp2(sc[u][e + 2] - m_use);
                    sum += sc[u][e] + sc[u][e + 2];
                }
                l_run[e] = l_run[e] * corr[e] + sum;
                m_ref[e] = m_new;
                refresh_any |= refresh;
            }
            if (__any_sync(0xffffffffu, refresh_any)) {
#pragma unroll
                for (int i = 0; i < C::kMt; ++i) {
                    acc[i][0] *= corr[0];
                    acc[i][1] *= corr[1];
                    acc[i][2] *= corr[0];
                    acc[i][3] *= corr[1];
                }
            }
            // ---- O^T += V^T (P s)^T ----------------------------------------------------------
#pragma unroll
            for (int st = 0; st < kSets; ++st) {
#pragma unroll
                for (int u = 0; u < C::kSub; ++u) {
                    const unsigned char *rows = tile + 16 * u * R::kBytes;
                    const unsigned char *x = rows + kr * R::kBytes, *y = x + 8 * R::kBytes;
                    const unsigned char *k0p = rows + kp * R::kBytes, *k1p = k0p + 2 * R::kBytes;
                    uint32_t px[kSet], py[kSet], q0[kSet], q1[kSet], q2[kSet], q3[kSet], ab[kSet], cd[kSet];
                    lds_words(px, x + R::kParamV + 4 * kSet * st);
                    lds_words(py, y + R::kParamV + 4 * kSet * st);
                    lds_words(q0, k0p + R::kParamV + 4 * kSet * st);
                    lds_words(q1, k1p + R::kParamV + 4 * kSet * st);
                    lds_words(q2, k0p + 8 * R::kBytes + R::kParamV + 4 * kSet * st);
                    lds_words(q3, k1p + 8 * R::kBytes + R::kParamV + 4 * kSet * st);
                    const int vo = R::kV + 2 * kSet * (8 * st + r);
                    v_pairs<kSet>(ab, k0p + vo, k1p + vo);
                    v_pairs<kSet>(cd, k0p + 8 * R::kBytes + vo, k1p + 8 * R::kBytes + vo);
#pragma unroll
                    for (int j = 0; j < kSet; ++j) {
                        const int g = st * kSet + j;
                        const float fx = q4_scale(px[j]), fy = q4_scale(py[j]);
                        uint32_t w0[kTerms], w1[kTerms];
                        split2<kTerms>(w0, sc[u][0] * fx, sc[u][1] * fx);
                        split2<kTerms>(w1, sc[u][2] * fy, sc[u][3] * fy);
                        const uint32_t b01 = __byte_perm(q0[j], q1[j], 0x7632), b23 = __byte_perm(q2[j], q3[j], 0x7632);
                        const uint32_t a0[4] = {q4_codes2(ab[j], 0, b01), q4_codes2(ab[j], 1, b01), q4_codes2(cd[j], 0, b23),
                                                q4_codes2(cd[j], 1, b23)};
                        const uint32_t a1[4] = {q4_codes2(ab[j], 2, b01), q4_codes2(ab[j], 3, b01), q4_codes2(cd[j], 2, b23),
                                                q4_codes2(cd[j], 3, b23)};
#pragma unroll
                        for (int k = kTerms - 1; k >= 0; --k) {
                            const uint32_t p0 = movmatrix_trans(w0[k]), p1 = movmatrix_trans(w1[k]);
                            mma_bf16_16816(acc[2 * g], a0, p0, p1);
                            if (2 * g + 1 < C::kMt) mma_bf16_16816(acc[2 * g + 1 < C::kMt ? 2 * g + 1 : 0], a1, p0, p1);
                        }
                    }
                }
            }
            if (valid < C::kKeys) fence_proxy_async_smem();  // the zeroed words precede the next copy
            __syncwarp();
            ++used;
            issue(known);
        }

        // ---- the end of a piece: the warps' states become one ---------------------------------
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l_run[e] += __shfl_xor_sync(0xffffffffu, l_run[e], 4);
            l_run[e] += __shfl_xor_sync(0xffffffffu, l_run[e], 8);
            l_run[e] += __shfl_xor_sync(0xffffffffu, l_run[e], 16);
        }
        if (lane < 4) {
            float *ml = sM + warp * 2 * kHeads;
            ml[2 * c] = m_ref[0];
            ml[2 * c + 1] = m_ref[1];
            ml[kHeads + 2 * c] = l_run[0];
            ml[kHeads + 2 * c + 1] = l_run[1];
        }
        __syncthreads();
        if (*abort_flag) break;  // seen by every thread alike: no wait lies between here and the barrier
        if (tid == 0) {          // one more piece for the table
            Walk w = *walk;
            if (known == 0 || !pieces[(known - 1) % kPieceRing].end) next_piece<TK>(a, w, HB, pieces[known % kPieceRing]);
            *walk = w;
        }
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < C::kWarps; ++w) M = fmaxf(M, sM[w * 2 * kHeads + 2 * c + e]);
            f[e] = fast_exp2(m_ref[e] - (M == -INFINITY ? 0.f : M));
        }
        const bool single = p.nseg == 1;
#pragma unroll
        for (int i0 = 0; i0 < C::kMt; i0 += C::kRound) {
            if (i0 > 0) __syncthreads();
            float *mine = park + warp * kHeads * C::kParkPitch;
#pragma unroll
            for (int i = 0; i < C::kRound; ++i)
                if (i0 + i < C::kMt) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        mine[(2 * c + (e & 1)) * C::kParkPitch + 16 * i + r + 8 * (e >> 1)] = acc[i0 + i][e] * f[e & 1];
                }
            __syncthreads();
            constexpr int kV4 = 4 * C::kRound;  // 4-channel vectors of a head in this round
            for (int v = tid; v < kHeads * kV4; v += C::kThreads) {
                const int h = v / kV4, x = 4 * (v % kV4), d = 16 * i0 + x;
                if (h >= g_cnt || d >= D) continue;
                float M = -INFINITY, l = 0.f;
#pragma unroll
                for (int w = 0; w < C::kWarps; ++w) M = fmaxf(M, sM[w * 2 * kHeads + h]);
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < C::kWarps; ++w) {
                    l += sM[w * 2 * kHeads + kHeads + h] * fast_exp2(sM[w * 2 * kHeads + h] - (M == -INFINITY ? 0.f : M));
                    const float4 t = *reinterpret_cast<const float4 *>(park + (w * kHeads + h) * C::kParkPitch + x);
                    o.x += t.x; o.y += t.y; o.z += t.z; o.w += t.w;
                }
                const float rl = 1.f / l;  // a piece holds a key: l > 0
                o.x *= rl; o.y *= rl; o.z *= rl; o.w *= rl;
                const int64_t bh = (int64_t)p.b * a.n_heads + h_base + h;
                const float lse2 = M + log2f(l);
                if (d == 0 && p.slot == 0) a.piece_count[bh] = p.nseg;
                if (single) {
                    T *dst = static_cast<T *>(a.out) + (int64_t)p.b * a.out_rs + (int64_t)(h_base + h) * D + d;
                    if constexpr (F32)
                        *reinterpret_cast<float4 *>(dst) = o;
                    else
                        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
                    if (d == 0 && a.lse != nullptr) a.lse[bh] = lse2 * kLn2;
                } else {
                    *reinterpret_cast<float4 *>(a.part_o + (bh * a.max_splits + p.slot) * D + d) = o;
                    if (d == 0) a.part_lse[bh * a.max_splits + p.slot] = lse2;
                }
            }
        }
        __syncthreads();  // the table has grown; sM, park and sQ are free
        if (!pieces[(known - 1) % kPieceRing].end) ++known;
        while (issued - used < (unsigned)C::kStages) {  // copies that had to wait for the table
            const unsigned before = issued;
            issue(known);
            if (issued == before) break;
        }
    }
    // every copy lands before the CTA leaves
    if (lane == 0) {
        volatile int no_abort = 0;
        const uint64_t until = globaltimer_ns() + 100000000ull;
        for (; used < issued; ++used)
            mbar_wait_bounded(&my_full[used % C::kStages], (used / C::kStages) & 1, &no_abort, until);
        if (warp == 0 && *abort_flag) report_status(a.status, kErrTimeout);
    }
}

template <int D, bool F32>
cudaError_t launch_q4_d(const Q4DecodeArgs &a, int grid, cudaStream_t s) {
    using C = Q4Cfg<D, F32>;
    cudaError_t e = cudaFuncSetAttribute(decode_q4_kernel<D, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    decode_q4_kernel<D, F32><<<grid, C::kThreads, C::kSmem, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const JoinArgs j{a.part_o, a.part_lse, a.piece_count, a.max_splits, a.n_heads, a.out, a.out_rs, a.lse};
    return launch_split_join<D, F32>(j, (int64_t)a.batch * a.n_heads, s);
}

template <int D, bool F32>
void shape_of(int *keys, int *tile, int *occ) {
    using C = Q4Cfg<D, F32>;
    *keys = C::kKeys;
    *tile = C::kTileKeys;
    static Occupancy occupancy;
    *occ = occupancy(decode_q4_kernel<D, F32>, C::kThreads, C::kSmem);
}

}  // namespace

bool plan_decode_q4(int batch, int n_heads, int n_kv_heads, int head_dim, bool bf16, int max_kv_len, int num_sms,
                    Q4Plan *p) {
    int tile = 0, occ = 0;
    switch (head_dim) {
        case 64: bf16 ? shape_of<64, false>(&p->box_rows, &tile, &occ) : shape_of<64, true>(&p->box_rows, &tile, &occ); break;
        case 80: bf16 ? shape_of<80, false>(&p->box_rows, &tile, &occ) : shape_of<80, true>(&p->box_rows, &tile, &occ); break;
        case 128: bf16 ? shape_of<128, false>(&p->box_rows, &tile, &occ) : shape_of<128, true>(&p->box_rows, &tile, &occ); break;
        case 256: bf16 ? shape_of<256, false>(&p->box_rows, &tile, &occ) : shape_of<256, true>(&p->box_rows, &tile, &occ); break;
        case 512: bf16 ? shape_of<512, false>(&p->box_rows, &tile, &occ) : shape_of<512, true>(&p->box_rows, &tile, &occ); break;
        default: return false;
    }
    const int G = n_heads / n_kv_heads, HB = (G + kHeads - 1) / kHeads;
    const int64_t units = (int64_t)batch * n_kv_heads * HB;
    // join grid: one CTA per (sequence, query head, up to 128 channels)
    if ((int64_t)batch * n_heads * ((head_dim + 127) / 128) > 0x7fffffffLL) return false;
    p->grid = num_sms * occ;
    // A unit of n tiles falls into at most n / min_tiles + 2 pieces.  min_tiles keeps that count
    // near 64 or, with few units, near the number of CTAs that each unit must feed.
    const int64_t range = ((int64_t)std::max(max_kv_len, 1) + tile - 1) / tile;
    const int64_t target = std::max<int64_t>(64, (p->grid + std::max<int64_t>(units, 1) - 1) / std::max<int64_t>(units, 1));
    p->min_tiles = (int)std::max<int64_t>(1, (range + target - 1) / target);
    p->max_splits = (int)((range + p->min_tiles - 1) / p->min_tiles) + 2;
    auto round256 = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t rows = (size_t)batch * n_heads;
    p->part_o_bytes = round256(rows * p->max_splits * head_dim * 4);
    p->part_lse_bytes = round256(rows * p->max_splits * 4);
    p->total_bytes = p->part_o_bytes + p->part_lse_bytes + round256(rows * 4);
    return true;
}

cudaError_t launch_decode_q4(const Q4DecodeArgs &a, bool bf16, int grid, cudaStream_t s) {
    switch (a.head_dim) {
        case 64: return bf16 ? launch_q4_d<64, false>(a, grid, s) : launch_q4_d<64, true>(a, grid, s);
        case 80: return bf16 ? launch_q4_d<80, false>(a, grid, s) : launch_q4_d<80, true>(a, grid, s);
        case 128: return bf16 ? launch_q4_d<128, false>(a, grid, s) : launch_q4_d<128, true>(a, grid, s);
        case 256: return bf16 ? launch_q4_d<256, false>(a, grid, s) : launch_q4_d<256, true>(a, grid, s);
        case 512: return bf16 ? launch_q4_d<512, false>(a, grid, s) : launch_q4_d<512, true>(a, grid, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace lat
