// decode_q8.cu — split-KV decode over an 8-bit KV cache (the record: q8_block.cuh).
//
// What it computes: for each sequence b and query head h, attention of one query row over the
// visible cached keys, key and value row j of block n read as s_n code_j, s_n = 2^e_n:
//   x_j = scale * s^K_n sum_d q_d k_jd    (then capped, if asked for)
//   out = sum_j e^{x_j - m} s^V_n v_j / sum_j e^{x_j - m}
//
// How:
//  * The stream of tiles, its shares and its joins: unit_stream.cuh.  Every warp is its own
//    pipeline: it owns kKeys rows of each tile; one bulk copy (of contiguous rows of a record) and
//    another of its 16 bytes of scales bring them into its ring, and its first lane issues those for a
//    stage as soon as the warp is done with it.  Warps meet only at the end of a piece.
//  * Both products run on mma m16n8k16 in fp16, where e4m3 codes are exact: one conversion
//    makes two codes an operand register.  Keys are M and heads N in the scores,
//    O^T[16 channels x 8 heads] += V^T P^T; the order of the channels within either product is
//    whatever puts a lane's codes side by side in the row.  V's pairs of keys come from two rows by
//    a byte permutation.
//  * A 16-key MMA tile lies in one block, so its scales are two numbers: K's joins the scores'
//    factor.  V's is a power of two and goes into the exponent of the weights:
//    w_j = 2^(x_j + e_n - r), r a running reference of x + e of its own, so that blocks of very
//    different size keep their weights in fp16's range; the sum of the softmax has its own
//    weights 2^(x_j - m), in fp32.  A weight is two fp16 terms, 2^-23 of it; the references lie
//    within 2^8 of the maxima and weights are taken 2^7 higher, so what falls under fp16's least is
//    2^-32 of the largest.  (One term, 2^-12 of a weight, moves one bf16 output in ten to the next
//    number: 8e-4 of the output, beside the 1.6e-3 of its rounding.  The second costs 0.5 % over long
//    caches, 8 x 131072 keys 300.8 -> 302.4 us, and 1 to 2 % on short ones: 32 ragged sequences of up
//    to 4096 keys 31.5 -> 31.8.)
//  * A query is brought to [2^8, 2^9) by a power of two of its own and taken as one fp16 number
//    (a bf16 channel above 2^-22 of the largest is exact) or, LAT_F32, two (22 bits and signs).
//  * LAT_F32: the scores' sums of 64 channels and the outputs' of 16 keys are chains of their own,
//    joined by rounded adds.  (8 x 131072 tokens, 32 heads over 8: 308 us, as without; head_dim 512
//    189 -> 210 us; the output's error 2.3e-6 -> 5e-7 of it over long caches.)  So are bf16's outputs up
//    to head_dim 128, where it is hidden behind HBM: 8 x 131072 keys 307.5 us, so 306.9, head_dim 64
//    160.6 -> 162.4, and the share of bf16 outputs that are the next number to the exact one's falls from 1 in
//    100 to next to none.  At head_dim 256 and 512 it would show, 312 -> 337 and 161 -> 181 us.
//  * Waits are bounded; on expiry the CTA records LAT_ERR_TIMEOUT, drains its copies, quits.
// What bounds it: HBM.  A 16-key tile of a warp is about 290 instructions at head_dim 128 for its
// 4 KB.  mma.sync rather than tcgen05: one query token fills 8 of N, and tcgen05 would need P in
// e4m3 terms, written to shared memory, for a kernel whose tensor pipe is busy 29 % of the time.
#include <algorithm>

#include "cache_kernels.h"
#include "device_common.cuh"
#include "f32x2.cuh"
#include "q8_block.cuh"
#include "score_cap.cuh"
#include "split_join.cuh"
#include "unit_stream.cuh"

namespace lat {

namespace {

constexpr float kWeightUp = 7.0f;  // log2: weights' place in fp16

template <int D, bool F32>
struct Q8Cfg {
    static constexpr int kWarps = 4;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kTerms = F32 ? 2 : 1;               // fp16 terms of q
    static constexpr int kWTerms = 2;                        // of a weight
    static constexpr bool kRounded = F32 || D <= 128;        // outputs' sums joined by rounded adds
    static constexpr int kRow = 2 * D;
    static constexpr int kSub = D <= 80 ? 4 : D == 512 ? 1 : 2;  // 16-key MMA tiles a warp takes at once
    static constexpr int kKeys = 16 * kSub;
    static constexpr int kTileKeys = kKeys * kWarps;
    static constexpr int kStages = 2;
    static constexpr int kScales = kKeys * kRow;             // where a stage's scales lie, 16 bytes a copy
    static constexpr int kStageBytes = kScales + 128;
    static constexpr int kMain = D / 64, kTail = D % 64 != 0;  // 64-channel runs; head_dim 80 has 16 more
    static constexpr int kSteps = D / 16;                    // MMAs of a score; 16-channel MMA tiles of O
    static constexpr bool kQReg = D < 512;                   // query fragments in registers, else in shared memory
    static constexpr int kRawRow = D * (F32 ? 4 : 2), kRawBytes = kHeads * kRawRow;
    static constexpr int kFragBytes = kQReg ? 0 : kSteps * 32 * 8 * kTerms;
    static constexpr int kQBytes = 2 * kRawBytes + kFragBytes;  // two units' queries as they are, fragments
    static constexpr int kRound = 8;                         // MMA tiles joined at once: 128 channels
    static constexpr int kParkPitch = 16 * kRound + 4;
    static constexpr int kParkBytes = kWarps * kHeads * kParkPitch * 4;
    static constexpr int kMinBlocks = D == 512 ? 1 : 2;      // CTAs per SM
    static constexpr int kMisc = 1024;
    static constexpr int kSmem = kWarps * kStages * kStageBytes + kQBytes + kParkBytes + kMisc;
    static_assert(kSmem <= 232448, "shared memory budget");
    static_assert(kSub * 16 <= 128, "scales of a stage");
};

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// two floats as TERMS packed fp16 pairs whose sum is the pair
template <int TERMS>
__device__ __forceinline__ void split_pair(uint32_t (&o)[TERMS], float x, float y) {
#pragma unroll
    for (int t = 0; t < TERMS; ++t) {
        o[t] = pack_f16x2(x, y);
        if (t + 1 < TERMS) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&o[t]));
            x -= f.x, y -= f.y;
        }
    }
}
__device__ __forceinline__ uint32_t f16_codes(uint32_t w, int half) { return e4m3x2_to_f16x2((uint16_t)(w >> (16 * half))); }

// d += the product of a with every term.
template <int TERMS>
__device__ __forceinline__ void mma_terms(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b0)[TERMS],
                                          const uint32_t (&b1)[TERMS]) {
#pragma unroll
    for (int t = TERMS - 1; t >= 0; --t) mma_f16_16816(d, a, b0[t], b1[t]);
}
// d += x, rounded.  The tensor pipe cuts a sum off where its last bit ends, always toward zero: along
// a chain of n products that is up to n 2^-23 of it, all to one side.  So long chains are short sums
// of their own, joined by these.
__device__ __forceinline__ void add_rounded(float (&d)[4], const float (&x)[4]) {
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
        const float2 s = halves_of(add2(pair_of(d[e], d[e + 1]), pair_of(x[e], x[e + 1])));
        d[e] = s.x, d[e + 1] = s.y;
    }
}

template <int D, bool F32>
__global__ void __launch_bounds__(Q8Cfg<D, F32>::kThreads, Q8Cfg<D, F32>::kMinBlocks)
decode_q8_kernel(const __grid_constant__ Q8DecodeArgs a) {
    using C = Q8Cfg<D, F32>;
    using T = typename std::conditional<F32, float, __nv_bfloat16>::type;
    constexpr int kTerms = C::kTerms, kWTerms = C::kWTerms, TK = C::kTileKeys;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char *ring = smem;                                              // [warp][stage]
    unsigned char *sQ = ring + C::kWarps * C::kStages * C::kStageBytes;      // raw queries, then fragments
    float *park = reinterpret_cast<float *>(sQ + C::kQBytes);                // [warp][head][channel]
    unsigned char *misc = reinterpret_cast<unsigned char *>(park) + C::kParkBytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(misc);                     // [warp][stage]
    float *sM = reinterpret_cast<float *>(misc + 128);                       // [warp][m[8], l[8]]
    StreamState &st = *reinterpret_cast<StreamState *>(misc + 384);
    Piece *pieces = st.pieces;
    volatile int *abort_flag = &st.abort_flag;
    static_assert(sizeof(StreamState) <= C::kMisc - 384, "misc area");

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.n_heads / a.n_kv_heads, HB = (G + kHeads - 1) / kHeads;
    auto prepare = [&] {
        for (int i = 0; i < C::kWarps * C::kStages; ++i) mbar_init(&full[i], 1);
        fence_mbarrier_init();
    };
    if (!stream_begin<TK, C::kKeys, C::kWarps, T>(a, HB, D, st, prepare)) return;
    const uint64_t deadline = globaltimer_ns() + a.timeout_ns;

    // ---- this warp's copies -------------------------------------------------------------
    unsigned char *my_ring = ring + warp * C::kStages * C::kStageBytes;
    uint64_t *my_full = full + warp * C::kStages;
    const int run_shift = min(a.block_shift, 31 - __clz(C::kKeys)), run = 1 << run_shift;  // rows of a copy
    int ip = 0, next = 0, keys = 0, from = 0;     // pieces taken up; next row and rows of the last one, its first key
    const unsigned char *at = nullptr;            // its head's records
    unsigned issued = 0, used = 0;                // stages issued, consumed
    // Issues this warp's next stage, if one is known.  `limit`: pieces in the table; `leave_out`:
    // the stage counts as issued and never comes.
    auto issue = [&](int limit, bool leave_out = false) {
        while (next >= keys) {
            if (ip >= limit) return;
            const Piece &p = pieces[ip % kPieceRing];
            if (p.end) return;
            ++ip;
            next = warp * C::kKeys;
            keys = p.keys, from = p.key0;
            at = a.cache + (int64_t)p.b * a.cache_seq + (int64_t)p.hk * a.cache_head;
        }
        if (lane == 0 && !leave_out) {
            const unsigned s = issued % C::kStages;
            unsigned char *to = my_ring + s * C::kStageBytes;
            const int runs = (min(C::kKeys, keys - next) + run - 1) >> run_shift;
            mbar_arrive_expect_tx(&my_full[s], runs * (run * C::kRow + 16));
            for (int i = 0; i < runs; ++i) {
                const int j = from + next + (i << run_shift);
                const unsigned char *rec = at + (int64_t)(j >> a.block_shift) * a.cache_block;
                bulk_load(to + i * run * C::kRow, rec + (j & ((1 << a.block_shift) - 1)) * C::kRow, run * C::kRow, &my_full[s]);
                bulk_load(to + C::kScales + 16 * i, rec + ((int64_t)C::kRow << a.block_shift), 16, &my_full[s]);
            }
        }
        ++issued;
        next += TK;
    };
    int known = 1;               // table entries written (or behind an end mark)
    int n_joins = 0;             // (thread 0)
    // A unit's queries come a unit ahead, so that they do not wait behind its rows
    const T *q_all = static_cast<const T *>(a.q);
    auto fetch_queries = [&](int i, int limit) {
        const Piece &n = pieces[i % kPieceRing];
        if (i < limit && !n.end) {
            const int h0 = n.hk * G + n.hb * kHeads, cnt = min(kHeads, G - n.hb * kHeads);
            const unsigned char *src = reinterpret_cast<const unsigned char *>(q_all + (int64_t)n.b * a.q_rs + (int64_t)h0 * D);
            for (int v = tid; v < cnt * (C::kRawRow / 16); v += C::kThreads)
                cp_async_16(sQ + (i & 1) * C::kRawBytes + 16 * v, src + 16 * v, true);
        }
        cp_async_commit();
    };
    fetch_queries(0, known);
    issue(known, a.test_skip_load);
    const bool missing = a.test_skip_load && issued > 0;  // test hook: the first stage is not there
    for (int s = 1; s < C::kStages; ++s) issue(known);
    auto one_more = [&]() {  // another entry for the table, by thread 0
        if (tid == 0 && !pieces[(known - 1) % kPieceRing].end) {
            Walk w = st.walk;
            next_piece<TK, C::kKeys>(a, w, HB, pieces[known % kPieceRing]);
            st.walk = w;
        }
    };
    one_more();
    cp_async_wait<0>();
    __syncthreads();
    if (!pieces[0].end) ++known;
    // fills the ring with what the table has
    auto issue_all = [&]() {
        while (issued - used < C::kStages) {
            const unsigned was = issued;
            issue(known);
            if (issued == was) break;
        }
    };
    issue_all();

    const int r = lane >> 2, c = lane & 3;
    for (int pi = 0;; ++pi) {
        const Piece p = pieces[pi % kPieceRing];
        if (p.end) break;
        const int h_base = p.hk * G + p.hb * kHeads, g_cnt = min(kHeads, G - p.hb * kHeads);
        // rows before this key are masked (the range begins on a multiple of kKeys)
        const int seen_from = a.window > 0 ? a.kv_lens[p.b] - a.window - p.key0 : 0;

        // ---- the unit's queries: lane (r, c) holds of head r the channels that its codes of
        // K will meet, four a step; hs brings the scores of heads 2 c and 2 c + 1 to the log2 domain
        uint32_t qf[C::kQReg ? C::kSteps : 1][2][kTerms];
        float hs[2], pre[2];
        {
            const unsigned char *raw = sQ + (pi & 1) * C::kRawBytes + r * C::kRawRow;
            auto channels = [&](int s, float (&v)[4]) {
                const int ch = s < 4 * C::kMain ? 16 * (c + 4 * (s >> 2)) + 4 * (s & 3) : 64 + 4 * c;
                if (r >= g_cnt) {
                    v[0] = v[1] = v[2] = v[3] = 0.f;
                } else if constexpr (F32) {
                    const float4 x = *reinterpret_cast<const float4 *>(raw + 4 * ch);
                    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
                } else {
                    const uint2 x = *reinterpret_cast<const uint2 *>(raw + 2 * ch);
                    v[0] = __uint_as_float(x.x << 16), v[1] = __uint_as_float(x.x & 0xffff0000u);
                    v[2] = __uint_as_float(x.y << 16), v[3] = __uint_as_float(x.y & 0xffff0000u);
                }
            };
            float m = 0.f;
#pragma unroll
            for (int s = 0; s < C::kSteps; ++s) {
                float v[4];
                channels(s, v);
#pragma unroll
                for (int k = 0; k < 4; ++k) m = larger_magnitude(m, fabsf(v[k]));
            }
            m = larger_magnitude(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = larger_magnitude(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const float by = to_f16_range(m, 8);
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // lane 4 h holds head h
                const float x = __shfl_sync(0xffffffffu, by, 8 * c + 4 * e);
                // 1 / x can exceed a float where the query is that large
                pre[e] = x < 0x1p-100f ? 0x1p20f : 1.f;
                hs[e] = (x < 0x1p-100f ? 0x1p-20f : 1.f) / x * a.scale_log2;
            }
            uint2 *frag = reinterpret_cast<uint2 *>(sQ + 2 * C::kRawBytes);  // [step][lane][term]
#pragma unroll
            for (int s = 0; s < C::kSteps; ++s) {
                if (!C::kQReg && s % C::kWarps != warp) continue;
                float v[4];
                uint32_t x[kTerms], y[kTerms];
                channels(s, v);
                split_pair<kTerms>(x, v[0] * by, v[1] * by);
                split_pair<kTerms>(y, v[2] * by, v[3] * by);
#pragma unroll
                for (int t = 0; t < kTerms; ++t) {
                    if constexpr (C::kQReg) qf[s][0][t] = x[t], qf[s][1][t] = y[t];
                    else frag[(s * 32 + lane) * kTerms + t] = make_uint2(x[t], y[t]);
                }
            }
            if constexpr (!C::kQReg) __syncthreads();
        }
        fetch_queries(pi + 1, known);
        // one more piece for the table, while the first tile is on its way
        one_more();
        // references of the scores and of scores plus V's exponents; the softmax's sum
        float m_ref[2] = {-INFINITY, -INFINITY}, v_ref[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
        float acc[C::kSteps][4];
#pragma unroll
        for (int i = 0; i < C::kSteps; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;

        for (int k0 = warp * C::kKeys; k0 < p.keys; k0 += TK) {
            const unsigned s = used % C::kStages;
            const bool got = mbar_wait_bounded(&my_full[s], (used / C::kStages) & 1, abort_flag, deadline);
            if (!__all_sync(0xffffffffu, got)) break;
            unsigned char *tile = my_ring + s * C::kStageBytes;
            const int valid = min(C::kKeys, p.keys - k0), hidden = max(0, seen_from - k0);
            const bool edge = valid < C::kKeys || hidden > 0;
            if (edge) {
                // rows that are not seen hold anything: zeros for their values, whose weights are
                // zero; scales of ones where nothing was copied
                for (int i = lane; i < C::kKeys * (D / 8); i += 32) {
                    const int row = i / (D / 8), off = D + i % (D / 8) * 8;
                    if (row < hidden || row >= valid)
                        *reinterpret_cast<uint2 *>(tile + row * C::kRow + q8_place<D>(off, row)) = make_uint2(0, 0);
                }
                if (lane < C::kSub && lane << run_shift >= valid)
                    *reinterpret_cast<float2 *>(tile + C::kScales + 16 * lane) = make_float2(1.f, 1.f);
                __syncwarp();
            }
            // ---- S^T ---------------------------------------------------------------------------
            float sc[C::kSub][4], v_exp[C::kSub];
#pragma unroll
            for (int u = 0; u < C::kSub; ++u) sc[u][0] = sc[u][1] = sc[u][2] = sc[u][3] = 0.f;
            auto query = [&](int step, uint32_t (&q)[2][kTerms]) {
                if constexpr (C::kQReg) {
#pragma unroll
                    for (int t = 0; t < kTerms; ++t) q[0][t] = qf[step][0][t], q[1][t] = qf[step][1][t];
                } else {
                    const uint2 *frag = reinterpret_cast<const uint2 *>(sQ + 2 * C::kRawBytes) + (step * 32 + lane) * kTerms;
#pragma unroll
                    for (int t = 0; t < kTerms; ++t) q[0][t] = frag[t].x, q[1][t] = frag[t].y;
                }
            };
            auto score_step = [&](float (&d)[4], uint32_t x, uint32_t y, int step) {
                const uint32_t k[4] = {f16_codes(x, 0), f16_codes(y, 0), f16_codes(x, 1), f16_codes(y, 1)};
                uint32_t q[2][kTerms];
                query(step, q);
                mma_terms<kTerms>(d, k, q[0], q[1]);
            };
#pragma unroll
            for (int u = 0; u < C::kSub; ++u) {
                const unsigned char *x = tile + (16 * u + r) * C::kRow, *y = x + 8 * C::kRow;
#pragma unroll
                for (int h = 0; h < C::kMain; ++h) {
                    const int off = q8_place<D>(16 * (c + 4 * h), r);
                    const uint4 wx = *reinterpret_cast<const uint4 *>(x + off), wy = *reinterpret_cast<const uint4 *>(y + off);
                    float x64[4] = {0.f, 0.f, 0.f, 0.f}, (&d)[4] = F32 ? x64 : sc[u];  // (of these 64 channels)
                    score_step(d, wx.x, wy.x, 4 * h);
                    score_step(d, wx.y, wy.y, 4 * h + 1);
                    score_step(d, wx.z, wy.z, 4 * h + 2);
                    score_step(d, wx.w, wy.w, 4 * h + 3);
                    if constexpr (F32) add_rounded(sc[u], x64);
                }
                if constexpr (C::kTail) {
                    const int off = 64 + 4 * c;
                    score_step(sc[u], *reinterpret_cast<const uint32_t *>(x + off), *reinterpret_cast<const uint32_t *>(y + off), 4);
                }
                const float2 scales = *reinterpret_cast<const float2 *>(tile + C::kScales + 16 * ((16 * u) >> run_shift));
                v_exp[u] = (float)((int)(__float_as_uint(scales.y) >> 23) - 127);
                // ---- the log2 domain, the cap, the mask ------------------------------------------
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    // (an infinity, of either sign, must not meet a score of 0)
                    const float f = fmaxf(fminf(hs[e] * scales.x, 3e38f), -3e38f);
                    sc[u][e] = sc[u][e] * pre[e] * f;
                    sc[u][e + 2] = sc[u][e + 2] * pre[e] * f;
                }
                if (a.cap_log2 > 0.f) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sc[u][e] = F32 ? a.cap_log2 * tanhf(sc[u][e] * a.over_cap_log2)
                                       : capped_score_close(sc[u][e] * a.over_cap_log2, a.cap_log2);
                }
                if (edge) {
                    const int i = 16 * u + r;
                    if (i >= valid || i < hidden) sc[u][0] = sc[u][1] = -INFINITY;
                    if (i + 8 >= valid || i + 8 < hidden) sc[u][2] = sc[u][3] = -INFINITY;
                }
            }
            // ---- running references and sum.  Any reference within 2^8 of its maximum serves; both
            // move (to the maxima) only when some score has outgrown one, which a vote tells --------
            float t[2], tv[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                t[e] = fmaxf(sc[0][e], sc[0][e + 2]);
                tv[e] = t[e] + v_exp[0];
#pragma unroll
                for (int u = 1; u < C::kSub; ++u) {
                    const float x = fmaxf(sc[u][e], sc[u][e + 2]);
                    t[e] = fmaxf(t[e], x);
                    tv[e] = fmaxf(tv[e], x + v_exp[u]);
                }
            }
            if (__any_sync(0xffffffffu, t[0] > m_ref[0] + kRescaleBy || t[1] > m_ref[1] + kRescaleBy ||
                                            tv[0] > v_ref[0] + kRescaleBy || tv[1] > v_ref[1] + kRescaleBy)) {
                float corr[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) {
                        t[e] = fmaxf(t[e], __shfl_xor_sync(0xffffffffu, t[e], off));
                        tv[e] = fmaxf(tv[e], __shfl_xor_sync(0xffffffffu, tv[e], off));
                    }
                    const float m_new = fmaxf(m_ref[e], t[e]), v_new = fmaxf(v_ref[e], tv[e]);
                    l_run[e] *= m_new == -INFINITY ? 1.f : fast_exp2(m_ref[e] - m_new);
                    corr[e] = v_new == -INFINITY ? 1.f : fast_exp2(v_ref[e] - v_new);
                    m_ref[e] = m_new;
                    v_ref[e] = v_new;
                }
#pragma unroll
                for (int i = 0; i < C::kSteps; ++i) {
                    acc[i][0] *= corr[0];
                    acc[i][1] *= corr[1];
                    acc[i][2] *= corr[0];
                    acc[i][3] *= corr[1];
                }
            }
            uint32_t w0[C::kSub][kWTerms], w1[C::kSub][kWTerms];
            {
                float m_use[2], v_use[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    m_use[e] = m_ref[e] == -INFINITY ? 0.f : m_ref[e];
                    v_use[e] = v_ref[e] == -INFINITY ? 0.f : v_ref[e] - kWeightUp;
                }
#pragma unroll
                for (int u = 0; u < C::kSub; ++u) {
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        w[e] = fast_exp2(sc[u][e] - (v_use[e & 1] - v_exp[u]));
                        l_run[e & 1] += fast_exp2(sc[u][e] - m_use[e & 1]);
                    }
                    split_pair<kWTerms>(w0[u], w[0], w[1]);
                    split_pair<kWTerms>(w1[u], w[2], w[3]);
#pragma unroll
                    for (int k = 0; k < kWTerms; ++k) w0[u][k] = movmatrix_trans(w0[u][k]), w1[u][k] = movmatrix_trans(w1[u][k]);
                }
            }
            // ---- O^T += V^T P^T: lane (r, c) takes channels of its own for rows 2 c, 2 c + 1, 2 c + 8
            // and 2 c + 9 of a tile; bytes 2 i and 2 i + 1 are rows r and r + 8 of MMA tile i --------
            auto add_product = [&](float (&d)[4], const uint32_t (&v)[4], int u) {
                if constexpr (C::kRounded) {
                    float x[4] = {0.f, 0.f, 0.f, 0.f};
                    mma_terms<kWTerms>(x, v, w0[u], w1[u]);
                    add_rounded(d, x);
                } else {
                    mma_terms<kWTerms>(d, v, w0[u], w1[u]);
                }
            };
#pragma unroll
            for (int u = 0; u < C::kSub; ++u) {
                const unsigned char *row[4];
                int sw[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int j = 2 * c + (k & 1) + 8 * (k >> 1);
                    row[k] = tile + (16 * u + j) * C::kRow;
                    sw[k] = j;
                }
                auto pair = [&](const uint32_t (&w)[4], int i) {  // four channels: MMA tiles i, i + 1
                    const uint32_t x0 = __byte_perm(w[0], w[1], 0x5140), y0 = __byte_perm(w[2], w[3], 0x5140);
                    const uint32_t x1 = __byte_perm(w[0], w[1], 0x7362), y1 = __byte_perm(w[2], w[3], 0x7362);
                    const uint32_t a0[4] = {f16_codes(x0, 0), f16_codes(x0, 1), f16_codes(y0, 0), f16_codes(y0, 1)};
                    const uint32_t a1[4] = {f16_codes(x1, 0), f16_codes(x1, 1), f16_codes(y1, 0), f16_codes(y1, 1)};
                    add_product(acc[i], a0, u);
                    add_product(acc[i + 1], a1, u);
                };
                if constexpr (D >= 128) {
#pragma unroll
                    for (int h = 0; h < D / 128; ++h) {
                        uint4 v[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) v[k] = *reinterpret_cast<const uint4 *>(row[k] + q8_place<D>(D + 16 * (r + 8 * h), sw[k]));
                        const uint32_t i0[4] = {v[0].x, v[1].x, v[2].x, v[3].x}, i1[4] = {v[0].y, v[1].y, v[2].y, v[3].y};
                        const uint32_t i2[4] = {v[0].z, v[1].z, v[2].z, v[3].z}, i3[4] = {v[0].w, v[1].w, v[2].w, v[3].w};
                        pair(i0, 8 * h);
                        pair(i1, 8 * h + 2);
                        pair(i2, 8 * h + 4);
                        pair(i3, 8 * h + 6);
                    }
                } else {
                    uint2 v[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = *reinterpret_cast<const uint2 *>(row[k] + q8_place<D>(D + 8 * r, sw[k]));
                    const uint32_t i0[4] = {v[0].x, v[1].x, v[2].x, v[3].x}, i1[4] = {v[0].y, v[1].y, v[2].y, v[3].y};
                    pair(i0, 0);
                    pair(i1, 2);
                    if constexpr (C::kTail) {  // channels 64 + 2 r and the next
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) w[k] = *reinterpret_cast<const uint16_t *>(row[k] + D + 64 + 2 * r);
                        const uint32_t x = __byte_perm(w[0], w[1], 0x5140), y = __byte_perm(w[2], w[3], 0x5140);
                        const uint32_t a0[4] = {f16_codes(x, 0), f16_codes(x, 1), f16_codes(y, 0), f16_codes(y, 1)};
                        add_product(acc[C::kSteps - 1], a0, u);
                    }
                }
            }
            if (edge) fence_proxy_async_smem();  // the zeroed words precede the next copy
            __syncwarp();
            ++used;
            issue(known);
        }

        // ---- the end of a piece: the warps' states become one ---------------------------------
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l_run[e] += __shfl_xor_sync(0xffffffffu, l_run[e], off);
        if (lane < 4) {
            float *ml = sM + warp * 2 * kHeads;
            ml[2 * c] = m_ref[0];
            ml[2 * c + 1] = m_ref[1];
            ml[kHeads + 2 * c] = l_run[0];
            ml[kHeads + 2 * c + 1] = l_run[1];
        }
        __syncthreads();
        if (*abort_flag) break;  // seen by every thread alike: no wait lies between here and the barrier
        // this warp's share of heads 2 c and 2 c + 1: its values' reference over the sum of all
        float f[2];
        const bool single = p.nseg == 1;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float M = -INFINITY, l = 0.f;
#pragma unroll
            for (int w = 0; w < C::kWarps; ++w) M = fmaxf(M, sM[w * 2 * kHeads + 2 * c + e]);
            const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int w = 0; w < C::kWarps; ++w)
                l = fmaf(sM[w * 2 * kHeads + kHeads + 2 * c + e], fast_exp2(sM[w * 2 * kHeads + 2 * c + e] - base), l);
            // (a piece whose scores are all below the least float has weight zero, not 0 / 0)
            f[e] = l == 0.f ? 0.f : fast_exp2(v_ref[e] - kWeightUp - base) / l;
            if (warp == 0 && r == 0 && 2 * c + e < g_cnt) {
                const int64_t bh = (int64_t)p.b * a.n_heads + h_base + 2 * c + e;
                const float lse2 = M + log2f(l);
                if (a.defer_join && p.slot == 0) a.piece_count[bh] = p.nseg;
                if (!single) a.part_lse[bh * a.max_splits + p.slot] = lse2;
                else if (a.lse != nullptr) a.lse[bh] = lse2 * kLn2;
            }
        }
#pragma unroll
        for (int i0 = 0; i0 < C::kSteps; i0 += C::kRound) {
            if (i0 > 0) __syncthreads();
            float *mine = park + warp * kHeads * C::kParkPitch;
#pragma unroll
            for (int i = 0; i < C::kRound; ++i)
                if (i0 + i < C::kSteps) {
                    // this lane's channels of MMA tile i0 + i, from 16 i0 on
                    const int ch = D >= 128 ? 16 * r + 2 * i : i < 4 ? 8 * r + 2 * i : 64 + 2 * r;
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *reinterpret_cast<float2 *>(mine + (2 * c + e) * C::kParkPitch + ch) =
                            make_float2(acc[i0 + i][e] * f[e], acc[i0 + i][e + 2] * f[e]);
                }
            __syncthreads();
            constexpr int kV4 = 4 * C::kRound;  // 4-channel vectors of a head in this round
            for (int v = tid; v < kHeads * kV4; v += C::kThreads) {
                const int h = v / kV4, x = 4 * (v % kV4), d = 16 * i0 + x;
                if (h >= g_cnt || d >= D) continue;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < C::kWarps; ++w) {
                    const float4 y = *reinterpret_cast<const float4 *>(park + (w * kHeads + h) * C::kParkPitch + x);
                    o.x += y.x; o.y += y.y; o.z += y.z; o.w += y.w;
                }
                if (single) {
                    T *dst = static_cast<T *>(a.out) + (int64_t)p.b * a.out_rs + (int64_t)(h_base + h) * D + d;
                    if constexpr (F32)
                        *reinterpret_cast<float4 *>(dst) = o;
                    else
                        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
                } else {
                    const int64_t bh = (int64_t)p.b * a.n_heads + h_base + h;
                    *reinterpret_cast<float4 *>(a.part_o + (bh * a.max_splits + p.slot) * D + d) = o;
                }
            }
        }
        cp_async_wait<0>();  // the next unit's queries
        __syncthreads();     // the table has grown; sM, park and sQ are free
        if (tid == 0 && !single && n_joins < 2)  // at most a CTA's first and last piece
            st.joins[n_joins++] = Join{p.b, h_base, g_cnt, p.nseg, (p.b * a.n_kv_heads + p.hk) * HB + p.hb, 0};
        if (!pieces[(known - 1) % kPieceRing].end) ++known;
        issue_all();
    }
    // every copy lands before the CTA leaves, a next unit's queries among them
    cp_async_wait<0>();
    if (lane == 0) {
        volatile int no_abort = 0;
        const uint64_t until = globaltimer_ns() + 100000000ull;
        if (missing && used == 0) ++used;
        for (; used < issued; ++used)
            mbar_wait_bounded(&my_full[used % C::kStages], (used / C::kStages) & 1, &no_abort, until);
        if (warp == 0 && *abort_flag) report_status(a.status, kErrTimeout);
    }
    stream_join<D, F32, C::kThreads>(a, st);
}

template <int D, bool F32>
cudaError_t launch_q8(const Q8DecodeArgs &a, int grid, cudaStream_t s) {
    using C = Q8Cfg<D, F32>;
    // (the plan's question for the occupancy has set the shared memory limit)
    decode_q8_kernel<D, F32><<<grid, C::kThreads, C::kSmem, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.defer_join) return e;
    const JoinArgs j{a.part_o, a.part_lse, a.piece_count, a.max_splits, a.n_heads, a.out, a.out_rs, a.lse};
    return launch_split_join<D, F32>(j, (int64_t)a.batch * a.n_heads, s);
}

// the grid, and the keys of a tile
template <int D, bool F32>
int shape_of(SplitPlan *p, int sms) {
    using C = Q8Cfg<D, F32>;
    static Occupancy occupancy;
    p->grid = sms * occupancy(decode_q8_kernel<D, F32>, C::kThreads, C::kSmem);
    return C::kTileKeys;
}

// calls f<D, F32> for a supported head_dim and type
#define LAT_Q8_CASE(D, bf16, f, ...) \
    case D: return (bf16) ? f<D, false>(__VA_ARGS__) : f<D, true>(__VA_ARGS__);
#define LAT_Q8_DISPATCH(head_dim, bf16, f, other, ...) \
    switch (head_dim) {                                \
        LAT_Q8_CASE(64, bf16, f, __VA_ARGS__)          \
        LAT_Q8_CASE(80, bf16, f, __VA_ARGS__)          \
        LAT_Q8_CASE(128, bf16, f, __VA_ARGS__)         \
        LAT_Q8_CASE(256, bf16, f, __VA_ARGS__)         \
        LAT_Q8_CASE(512, bf16, f, __VA_ARGS__)         \
        default: return other;                         \
    }
int shape(int head_dim, bool bf16, SplitPlan *p, int sms) { LAT_Q8_DISPATCH(head_dim, bf16, shape_of, 0, p, sms) }

}  // namespace

bool plan_decode_q8(int batch, int n_heads, int n_kv_heads, int head_dim, bool bf16, int max_kv_len, int num_sms,
                    SplitPlan *p) {
    const int G = n_heads / n_kv_heads, HB = (G + kHeads - 1) / kHeads;
    const int tile = shape(head_dim, bf16, p, num_sms);
    if (tile == 0) return false;
    return plan_units(p, (int64_t)batch * n_kv_heads * HB, ((int64_t)std::max(max_kv_len, 1) + tile - 1) / tile,
                      (int64_t)batch * n_heads, head_dim);
}

cudaError_t launch_decode_q8(const Q8DecodeArgs &a, bool bf16, const SplitPlan &p, cudaStream_t s) {
    LAT_Q8_DISPATCH(a.head_dim, bf16, launch_q8, cudaErrorInvalidValue, a, p.grid, s)
}

}  // namespace lat
