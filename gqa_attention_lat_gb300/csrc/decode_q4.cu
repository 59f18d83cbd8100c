// decode_q4.cu — split-KV decode over a 4-bit KV cache (the row format: q4_row.cuh).
//
// What it computes: for each sequence b and query head h, attention of one query row over
// the visible cached keys, with key and value channel d of group g read as s_jg (c_jd - z_jg):
//   x_j = scale * sum_g s_jg sum_{d in g} q_d (c_jd - z_jg)      (then capped, if asked for)
//   out = sum_j e^{x_j - m} v_j / sum_j e^{x_j - m}
// The scale never meets the codes: a group's products are summed by the tensor cores and
// scaled once per key, and V's scales multiply the softmax weights, p_j s_jg, before
// two bf16 terms are made of them.
//
// How:
//  * Work unit = one (sequence, KV head, block of <= 8 query heads).  All units' keys, laid
//    end to end in tiles of kTileKeys, form one stream; CTA c takes the c-th equal share
//    (to a tile, never under min_tiles).  A unit cut across CTAs leaves one normalised partial and its
//    log-sum-exp per piece.  The CTA that finishes a unit's last piece (an atomic ticket) joins
//    them after its stream; units of many pieces are joined by a second kernel instead (a
//    programmatic dependent), which spreads a head's channels over CTAs.
//  * Every warp is its own pipeline: it owns kKeys rows of each tile, which one TMA copy
//    brings into its ring (a box over the cache's strides; the row is one run of bytes for
//    K and V), and its first lane issues the copy for a stage as soon as the warp is done
//    with it.  Warps meet only at the end of a piece.
//  * Scores on mma m16n8k16 in fp16, keys in M, heads in N, by groups of 32 channels: a nibble
//    left where it lies in the low byte of a half, ORed into fp16 2^-10, is 2^-20 times 1024 + c
//    or 16 (64 + c); 2^-20 times 960 less brings the first to 64 + c too, exactly.  So a word of
//    codes is four operand registers for four AND-ORs, a shift and two subtractions, and the
//    query's channels on the 16-fold codes are taken 16 times smaller.  The zero point enters as
//    (64 + z) times the group's sum of the query.  An MMA lines its products up by the exponents
//    that the operands carry: the bare codes as fp16 subnormals need neither OR nor subtraction,
//    but lost six bits (log-sum-exp 2e-6 off, against 1e-7 now).  Taking off 8 from every nibble
//    instead gave 5e-8, for 280 instead of 273 us on 8 x 131072 keys at the time.  A query is
//    brought to [2^8, 2^9) by a power of two of its own: channels above 2^-20 of its largest stay
//    exact, smaller ones are within 2^-29 of it.
//  * O^T[16 channels x 8 heads] += V^T (P s)^T on mma m16n8k16 in bf16 (a weight needs bf16's
//    range): a nibble becomes 128 + c by an AND-OR (0x4300 is bf16 128, whose last place is 1),
//    minus 128 + z, exactly.  The rows' layout puts a lane's codes side by side.  A weight is
//    two bf16 terms (16 bits): with one, its rounding was as large as the bf16 output's own
//    (2.2e-3 off in all where the output's alone is 1.6e-3).  Units of up to 4 heads (Twin) have
//    their heads twice in N, columns 0-3 with the first terms and 4-7 with the second, and add the
//    two halves up at a piece's end; others take a second MMA (8 x 131072 keys, 4 heads a KV
//    head: one term 234 us, twice in N 249, two MMAs 274; 8 heads a KV head: 275).
//  * LAT_F32: the query is two fp16 terms (22 bits and their signs, 2^-24 of a channel), the
//    codes lose their zero point before the product, and the weights p s are three bf16 terms.
//  * Waits are bounded; on expiry the CTA records LAT_ERR_TIMEOUT, drains its copies, quits.
// What bounds it: the logic pipe.  A warp instruction takes it two cycles of an SM's four
// schedulers (measured: LOP3, PRMT and conversions 2 a cycle and SM, fp16 and bf16 MMA 0.49; an
// e4m3 MMA, which would take the codes as they are, is unpacked to fp16 by 12 conversions here).
#include <math.h>

#include <algorithm>

#include <cuda_fp16.h>

#include "cache_kernels.h"
#include "device_common.cuh"
#include "q4_row.cuh"
#include "score_cap.cuh"
#include "split_join.cuh"

namespace lat {

namespace {

constexpr int kHeads = 8;                  // N of the mma: query heads of a unit
constexpr int kTwinHeads = 4;              // heads of a unit that fill N twice
constexpr float kRescaleBy = 8.0f;         // log2 units the maximum may grow unnoticed
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kPieceRing = 8;              // pieces known ahead
// What a unit costs beside its tiles (its queries made ready, the warps' states joined), in
// tiles: counted in the shares, so that a CTA of many short units is not the last to finish (32
// sequences of 1 to 4096 keys: not counted 36.8 us, as 2 tiles 30.5 us).
constexpr int kUnitCost = 2;

// The more keys a warp takes at once, the further a tile's fixed costs spread, until its registers
// cost CTAs (8 x 131072 keys, 16 times kSub keys: head_dim 64 2 163 us, 3 152, 4 143; 80 2 209,
// 3 198, 4 200; 256 2 479, 3 876).  At head_dim 128 that comes with tiles too coarse for short
// units, so there are two forms; kWideKeys says when.  (fp32 queries there gain nothing.)
template <int D, bool F32>
constexpr bool kHasWide = D == 128 && !F32;
template <int D, bool F32, bool Wide, bool Twin>
struct Q4Cfg {
    using R = Q4Row<D>;
    static constexpr int kWarps = 4;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kTerms = F32 ? 3 : Twin ? 1 : 2;    // bf16 terms of p s in MMAs of their own
    static constexpr int kQTerms = F32 ? 2 : 1;              // fp16 terms of q
    static constexpr float kUnit = F32 ? 0x1p-24f : 0x1p-20f;  // of the scores' products
    static constexpr int kQTo = F32 ? 12 : 8;                // its largest channel's exponent
    static constexpr int kSub = D == 64 || Wide ? 4 : D == 80 ? 3 : D == 512 ? 1 : 2;  // 16-key MMA tiles a warp takes at once
    static constexpr int kKeys = 16 * kSub;
    static constexpr int kTileKeys = kKeys * kWarps;
    static constexpr int kStages = 2;
    static constexpr int kStageBytes = kKeys * R::kBytes;
    // Rows of whole 128-byte pieces (head_dim 80: one, 512: five) would all begin in the same
    // bank.  Their copies lay each piece of the kKeys rows behind the last and permute its 16-byte
    // parts by the row's number (the 128-byte swizzle: part p of row j lies at p ^ (j % 8)).
    static constexpr bool kSwizzle = R::kBytes % 128 == 0;
    static constexpr int kPitch = kSwizzle ? 128 : R::kBytes;
    // where byte `off` of a row lies from its first; x: 16 (row % 8)
    static __device__ __forceinline__ int place(int off, int x) {
        return kSwizzle ? (off >> 7) * (kKeys * 128) + ((off & 127) ^ x) : off;
    }
    static constexpr int kMt = D / 16;                       // 16-channel MMA tiles
    static constexpr bool kQReg = R::kPad * kQTerms <= 256;  // query fragments in registers
    // else in shared memory: [term][head] rows of 16 bytes an octet, 16 words apart in the banks,
    // [group][head] sums, [head] factors
    static constexpr int kQRow = 2 * R::kPad + 64;
    // (in registers: two units' queries as they are, this one's and the next's)
    static constexpr int kRawRow = D * (F32 ? 4 : 2), kRawBytes = kHeads * kRawRow;
    static constexpr int kQBytes = kQReg ? 2 * kRawBytes : kQTerms * kHeads * kQRow + (R::kGroups + 1) * kHeads * 4;
    static constexpr int kRound = 8;                         // MMA tiles joined at once: 128 channels
    static constexpr int kParkPitch = 16 * kRound + 4;
    static constexpr int kParkBytes = kWarps * kHeads * kParkPitch * 4;
    static constexpr int kMinBlocks = D == 512 ? 1 : D == 256 || Wide || (D == 128 && F32) ? 2 : 3;  // CTAs per SM
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

struct Join {          // a unit cut across CTAs that this one may have to join
    int b, h_base, g_cnt, nseg, unit, last;
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

// The stream of `total` tiles in equal shares: the first `more` CTAs have each + 1, the others each
struct Shares {
    uint32_t each, more;
    __device__ __forceinline__ uint32_t begin(uint32_t c) const { return each * c + min(c, more); }
    __device__ __forceinline__ uint32_t of(uint32_t x) const {  // whose tile x is
        const uint32_t b = more * (each + 1);
        return x < b ? x / (each + 1) : more + (x - b) / each;
    }
};
// thread 0's place in the stream
struct Walk {
    uint32_t pos, end, pb;  // pb: where sequence b's units begin
    Shares shares;
    int b;
};

// a unit of n keys in the stream: nothing, or its tiles and what it costs beside them; where no
// unit is to be cut (a.whole), as much as the longest
template <int T>
__device__ __forceinline__ uint32_t tiles_of(int n) {
    return ((uint32_t)n + (T - 1)) / T;
}
template <int T>
__device__ __forceinline__ uint32_t unit_cost(const Q4DecodeArgs &a, int n) {
    return n <= 0 ? 0u : a.whole ? (uint32_t)a.min_tiles : tiles_of<T>(n) + kUnitCost;
}
template <int T>
__device__ bool next_piece(const Q4DecodeArgs &a, Walk &w, int HB, Piece &p) {
    const uint32_t HU = (uint32_t)(a.n_kv_heads * HB);
    while (w.pos < w.end && w.b < a.batch) {
        const KeyRange k = range_of(a, a.kv_lens[w.b]);
        const uint32_t cost = unit_cost<T>(a, k.n), nt = tiles_of<T>(k.n), all = cost * HU;
        if (w.pos >= w.pb + all) {
            w.pb += all;
            ++w.b;
            continue;
        }
        const uint32_t idx = (w.pos - w.pb) / cost, ustart = w.pb + idx * cost + kUnitCost;  // its first tile
        const uint32_t uend = ustart + nt;                                                       // behind its last
        const uint32_t t0 = w.pos > ustart ? w.pos - ustart : 0, t1 = w.end > ustart ? min(nt, w.end - ustart) : 0;
        const bool cut = w.pos > ustart;  // (divisions only for units that leave this share)
        w.pos = min(w.end, w.pb + (idx + 1) * cost);
        if (t0 >= t1) continue;  // the share ends before the unit's first tile
        const uint32_t first = cut ? w.shares.of(ustart) : blockIdx.x, last = uend > w.end ? w.shares.of(uend - 1) : blockIdx.x;
        p.b = w.b;
        p.hk = HB == 1 ? (int)idx : (int)(idx / HB);
        p.hb = HB == 1 ? 0 : (int)(idx % HB);
        p.key0 = k.lo + (int)t0 * T;
        p.keys = (int)(min((uint32_t)k.n, t1 * T) - t0 * T);
        p.slot = (int)(blockIdx.x - first);
        p.nseg = (int)(last - first + 1);
        p.end = 0;
        return true;
    }
    p.end = 1;
    return false;
}

// N consecutive 32-bit words at byte `off` of a row, in the widest loads their count allows
template <typename C, int N>
__device__ __forceinline__ void lds_words(uint32_t (&w)[N], const unsigned char *row, int off, int x) {
    if constexpr (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(row + C::place(off, x));
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(row + C::place(off, x));
        w[0] = v.x, w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = *reinterpret_cast<const uint32_t *>(row + C::place(off + 4 * i, x));
    }
}
// a lane's V halves of one set from two rows, paired: low halves from row r0, high from row r1
template <typename C, int SET>
__device__ __forceinline__ void v_pairs(uint32_t (&u)[SET], const unsigned char *r0, const unsigned char *r1, int off,
                                        int x0, int x1) {
    if constexpr (SET % 2 == 0) {
        uint32_t wx[SET / 2], wy[SET / 2];
        lds_words<C>(wx, r0, off, x0);
        lds_words<C>(wy, r1, off, x1);
#pragma unroll
        for (int j = 0; j < SET; ++j) u[j] = __byte_perm(wx[j / 2], wy[j / 2], (j & 1) ? 0x7632 : 0x5410);
    } else {
#pragma unroll
        for (int j = 0; j < SET; ++j)
            u[j] = (uint32_t)*reinterpret_cast<const uint16_t *>(r0 + C::place(off + 2 * j, x0)) |
                   ((uint32_t)*reinterpret_cast<const uint16_t *>(r1 + C::place(off + 2 * j, x1)) << 16);
    }
}

// an octet of a query as TERMS fp16 operands: channels 0, 1 and 4, 5 as they are, 2, 3 and 6, 7
// a sixteenth, in the order of the two MMAs' B registers
template <int TERMS>
__device__ __forceinline__ void split_f16(uint32_t (&o)[TERMS][4], const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a = x[2 * i], b = x[2 * i + 1];
        if (i & 1) a *= 0.0625f, b *= 0.0625f;
#pragma unroll
        for (int t = 0; t < TERMS; ++t) {
            const __half2 h = __floats2half2_rn(a, b);
            o[t][i] = *reinterpret_cast<const uint32_t *>(&h);
            if (t + 1 < TERMS) {
                const float2 f = __half22float2(h);
                a -= f.x, b -= f.y;
            }
        }
    }
}
// the power of two that brings m >= 0 to [2^to, 2^(to + 1)), as near as floats have one; 1 for
// nothing, NaN for what is not finite
__device__ __forceinline__ float to_f16_range(float m, int to) {
    const int e = (int)(__float_as_uint(m) >> 23);
    if (e == 255) return NAN;
    return m == 0.f ? 1.f : __uint_as_float((uint32_t)max(1, min(254, 127 + to + 127 - e)) << 23);
}
__device__ __forceinline__ uint32_t hsub2_f16(uint32_t x, uint32_t y) {
    const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&y));
    return *reinterpret_cast<const uint32_t *>(&d);
}
// nibbles at bits 0 or 4 (`shift`) of a word's halves in the last places of kOr, a pair of fp16,
// less another (0 for none)
template <uint32_t kOr>
__device__ __forceinline__ uint32_t f16_codes(uint32_t w, int shift, uint32_t bias) {
    const uint32_t x = and_or(w, 0x000f000fu << shift, kOr);
    return bias ? hsub2_f16(x, bias) : x;
}
// a parameter word's z as fp16 1024 + (z << shift), twice
__device__ __forceinline__ uint32_t f16_bias(uint32_t w, int shift) {
    return ((((w >> 16) & 0xfu) * 0x00010001u) << shift) | 0x64006400u;
}
__device__ __forceinline__ void mma_f16_16816(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ int add_acq_rel(int32_t *p, int x) {
    int was;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(was) : "l"(p), "r"(x) : "memory");
    return was;
}

// x and y plus `by` (a bf16) times the halves of a bf16 pair, without unpacking it (the logic
// pipe's work)
__device__ __forceinline__ void add_pair(float &x, float &y, uint32_t pair, uint16_t by) {
    asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\n"
        "fma.rn.f32.bf16 %0, l, %3, %0;\nfma.rn.f32.bf16 %1, h, %3, %1;\n}"
        : "+f"(x), "+f"(y) : "r"(pair), "h"(by));
}
constexpr uint16_t kMinusOne = 0xbf80u;  // in bf16
// two floats as `TERMS` packed bf16 pairs whose sum is the pair (to 8 bits a term)
template <int TERMS>
__device__ __forceinline__ void split2(uint32_t (&o)[TERMS], float x, float y) {
#pragma unroll
    for (int t = 0; t < TERMS; ++t) {
        o[t] = pack_bf16x2(x, y);
        if (t + 1 < TERMS) add_pair(x, y, o[t], kMinusOne);
    }
}
// the first term of both (by 0) or the second (by -1)
__device__ __forceinline__ uint32_t term2(float x, float y, uint16_t by) {
    add_pair(x, y, pack_bf16x2(x, y), by);
    return pack_bf16x2(x, y);
}

template <int D, bool F32, bool Wide, bool Twin>
__global__ void __launch_bounds__(Q4Cfg<D, F32, Wide, Twin>::kThreads, Q4Cfg<D, F32, Wide, Twin>::kMinBlocks)
decode_q4_kernel(const __grid_constant__ Q4DecodeArgs a) {
    using C = Q4Cfg<D, F32, Wide, Twin>;
    using R = Q4Row<D>;
    using T = typename std::conditional<F32, float, __nv_bfloat16>::type;
    constexpr int kTerms = C::kTerms, kQTerms = C::kQTerms, kSet = R::kSet, kSets = R::kGroups / R::kSet;
    extern __shared__ __align__(1024) unsigned char smem[];  // (an aligned-up pointer would load as generic)
    unsigned char *ring = smem;                                              // [warp][stage]
    unsigned char *sQ = ring + C::kWarps * C::kStages * C::kStageBytes;      // [term][head] rows
    float *park = reinterpret_cast<float *>(sQ + C::kQBytes);                // [warp][head][channel]
    unsigned char *misc = reinterpret_cast<unsigned char *>(park) + C::kParkBytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(misc);                     // [warp][stage]
    Piece *pieces = reinterpret_cast<Piece *>(misc + 128);                   // [kPieceRing]
    float *sM = reinterpret_cast<float *>(misc + 384);                       // [warp][m[8], l[8]]
    Walk *walk = reinterpret_cast<Walk *>(misc + 640);
    uint32_t *scan = reinterpret_cast<uint32_t *>(misc + 704);               // [warps]
    volatile int *abort_flag = reinterpret_cast<int *>(misc + 768);
    Join *joins = reinterpret_cast<Join *>(misc + 784);                      // [2]
    static_assert(sizeof(Piece) * kPieceRing <= 256 && sizeof(Walk) <= 64 && sizeof(Join) * 2 <= 64, "misc area");

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.n_heads / a.n_kv_heads, HB = (G + kHeads - 1) / kHeads, HU = a.n_kv_heads * HB;
    constexpr int TK = C::kTileKeys;

    // ---- the stream's length in tiles and this CTA's share: per-thread sums over a slice of
    // the sequences, then a scan ----------------------------------------------------------
    const int per_thread = (a.batch + C::kThreads - 1) / C::kThreads;
    const int b_lo = min(a.batch, tid * per_thread), b_hi = min(a.batch, b_lo + per_thread);
    uint32_t my_sum = 0;
    for (int b = b_lo; b < b_hi; ++b) {
        const int len = a.kv_lens[b];
        const KeyRange k = range_of(a, len);
        my_sum += unit_cost<TK>(a, k.n) * HU;
        if (blockIdx.x == 0 && k.n == 0) {  // nothing to stream
            const bool bad = len < 0 || len > a.max_kv_len;
            if (bad) report_status(a.status, kErrBounds);
            for (int h = 0; h < a.n_heads; ++h) {
                if (a.defer_join) a.piece_count[(int64_t)b * a.n_heads + h] = 0;
                if (!bad && a.lse != nullptr) a.lse[(int64_t)b * a.n_heads + h] = -INFINITY;
            }
            if (!bad)
                for (int i = 0; i < a.n_heads * D; ++i) static_cast<T *>(a.out)[(int64_t)b * a.out_rs + i] = T(0.f);
        }
    }
    uint32_t incl = my_sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
    }
    if (lane == 31) scan[warp] = incl;
    if (tid == 0) {
        walk->pos = 0;
        walk->end = 0;
        walk->b = a.batch;
        for (int i = 0; i < C::kWarps * C::kStages; ++i) mbar_init(&full[i], 1);
        *abort_flag = 0;
        joins[0].nseg = joins[1].nseg = joins[0].last = joins[1].last = 0;
        fence_mbarrier_init();
        if (a.max_kv_len > 0) tma_prefetch_desc(&a.tm);  // (else there is none)
    }
    __syncthreads();
    uint32_t total = 0, my_start = incl - my_sum;
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w) {
        const uint32_t v = scan[w];
        if (w < warp) my_start += v;
        total += v;
    }
    const uint32_t parts = max(1u, min(gridDim.x, total / (uint32_t)a.min_tiles)), each = total / parts;
    const Shares shares{each, total - each * parts};
    const uint32_t r0 = blockIdx.x < parts ? shares.begin(blockIdx.x) : 0;
    const uint32_t r1 = blockIdx.x < parts ? shares.begin(blockIdx.x + 1) : 0;
    if (r0 < r1 && r0 >= my_start && r0 - my_start < my_sum) {  // the share begins in this slice
        uint32_t p = my_start;
        int b = b_lo;
        for (; b < b_hi; ++b) {
            const uint32_t w = unit_cost<TK>(a, range_of(a, a.kv_lens[b]).n) * HU;
            if (r0 < p + w) break;
            p += w;
        }
        Walk w{r0, r1, p, shares, b};
        next_piece<TK>(a, w, HB, pieces[0]);
        *walk = w;
    }
    if (a.defer_join) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (r0 >= r1) return;
    __syncthreads();
    const uint64_t deadline = globaltimer_ns() + a.timeout_ns;

    // ---- this warp's copies -------------------------------------------------------------
    unsigned char *my_ring = ring + warp * C::kStages * C::kStageBytes;
    uint64_t *my_full = full + warp * C::kStages;
    int ip = 0, next = 0, keys = 0;               // pieces taken up; next row and rows of the last one
    int from = 0, at_hk = 0, at_b = 0;            // its first key and place
    unsigned issued = 0, used = 0;                // copies issued, consumed
    // Issues this warp's next copy, if one is known.  `limit`: pieces in the table; `leave_out`:
    // the copy counts as issued and never comes.
    auto issue = [&](int limit, bool leave_out = false) {
        while (next >= keys) {
            if (ip >= limit) return;
            const Piece &p = pieces[ip % kPieceRing];
            if (p.end) return;
            ++ip;
            next = warp * C::kKeys;
            keys = p.keys, from = p.key0, at_hk = p.hk, at_b = p.b;
        }
        if (lane == 0 && !leave_out) {
            const unsigned s = issued % C::kStages;
            mbar_arrive_expect_tx(&my_full[s], C::kStageBytes);
            if constexpr (C::kSwizzle)
                tma_load_5d(my_ring + s * C::kStageBytes, &a.tm, &my_full[s], 0, from + next, 0, at_hk, at_b);
            else
                tma_load_4d(my_ring + s * C::kStageBytes, &a.tm, &my_full[s], 0, at_hk, from + next, at_b);
        }
        ++issued;
        next += TK;
    };
    int known = 1;               // table entries written (or behind an end mark)
    int n_joins = 0;             // (thread 0)
    // A unit's queries come a unit ahead: asked for after the copies of its rows, they would wait
    // behind them (2.5 us where they take 1).
    const T *q_all = static_cast<const T *>(a.q);
    auto fetch_queries = [&](int i, int limit) {
        if constexpr (C::kQReg) {
            const Piece &n = pieces[i % kPieceRing];
            if (i < limit && !n.end) {
                const int h0 = n.hk * G + n.hb * kHeads, cnt = min(kHeads, G - n.hb * kHeads);
                const unsigned char *src = reinterpret_cast<const unsigned char *>(q_all + (int64_t)n.b * a.q_rs + (int64_t)h0 * D);
                for (int v = tid; v < cnt * (C::kRawRow / 16); v += C::kThreads)
                    cp_async_16(sQ + (i & 1) * C::kRawBytes + 16 * v, src + 16 * v, true);
            }
            cp_async_commit();
        }
    };
    fetch_queries(0, known);
    issue(known, a.test_skip_load);
    const bool missing = a.test_skip_load && issued > 0;  // test hook: the first copy is not there
    for (int s = 1; s < C::kStages; ++s) issue(known);
    auto one_more = [&]() {  // another entry for the table, by thread 0
        if (tid == 0 && !pieces[(known - 1) % kPieceRing].end) {
            Walk w = *walk;
            next_piece<TK>(a, w, HB, pieces[known % kPieceRing]);
            *walk = w;
        }
    };
    one_more();
    cp_async_wait<0>();
    __syncthreads();
    if (!pieces[0].end) ++known;
    auto issue_all = [&]() {  // what had to wait for the table
        while (issued - used < (unsigned)C::kStages) {
            const unsigned before = issued;
            issue(known);
            if (issued == before) break;
        }
    };
    issue_all();

    const int r = lane >> 2, c = lane & 3;
    // MMA row r is the tile's key perm(r): the two low bits swapped, so that the eight lanes of
    // a 16-byte shared-memory access fall into different banks at a 160-byte row
    const int kr = (r & 4) | ((r & 1) << 1) | ((r >> 1) & 1);
    const int kp = ((c & 2) << 1) | (c & 1);  // perm(2 c); perm(2 c + 1) is kp + 2
    const int sw_r = kr << 4, sw_0 = kp << 4, sw_1 = (kp + 2) << 4;  // those rows' swizzles
    const uint16_t twin_by = c < 2 ? 0 : kMinusOne;                 // Twin: the term of this lane's columns

    for (int pi = 0;; ++pi) {
        const Piece p = pieces[pi % kPieceRing];
        if (p.end) break;
        const int h_base = p.hk * G + p.hb * kHeads, g_cnt = min(kHeads, G - p.hb * kHeads);
        // ---- the unit's queries: lane (r, c) holds head r's channels 32 g + 8 c .. + 7 -----
        // qz[g]: the sums of heads 2 c and 2 c + 1, in units of kUnit (F32 has no use for them); pre
        // and hs bring those heads' scores to the log2 domain: 1 / kUnit over the query's power of
        // two, which can exceed a float, and the scale.
        uint32_t qf[C::kQReg ? R::kGroups : 1][kQTerms][4];
        float qz[C::kQReg ? R::kGroups : 1][2];
        float hs[2], pre[2];
        auto undo = [&](int e, float by) {
            pre[e] = by < 0x1p-100f ? 1.f / C::kUnit : 1.f;
            hs[e] = (by < 0x1p-100f ? 1.f : 1.f / C::kUnit) / by * a.scale_log2;
        };
        const T *qrow = q_all + (int64_t)p.b * a.q_rs + (int64_t)h_base * D;
        constexpr int kRaw = F32 ? 2 : 1;  // 16-byte words of an octet
        auto load = [&](int column, int d, uint4 (&x)[kRaw]) {
            const int head = Twin ? column % kTwinHeads : column;
            const uint4 *src = C::kQReg ? reinterpret_cast<const uint4 *>(sQ + (pi & 1) * C::kRawBytes + head * C::kRawRow + d * (int)sizeof(T))
                                        : reinterpret_cast<const uint4 *>(qrow + (int64_t)head * D + d);
#pragma unroll
            for (int k = 0; k < kRaw; ++k) x[k] = head < g_cnt && d < D ? src[k] : make_uint4(0, 0, 0, 0);
        };
        auto octet = [](const uint4 (&x)[kRaw], float (&v)[8]) {
            if constexpr (F32) {
                const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[kRaw - 1].x, x[kRaw - 1].y, x[kRaw - 1].z, x[kRaw - 1].w};
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(w[k]);
            } else {
                const uint32_t w[4] = {x[0].x, x[0].y, x[0].z, x[0].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[2 * k] = __uint_as_float(w[k] << 16);
                    v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
                }
            }
        };
        auto larger = [](float x, float y) {  // of two magnitudes, by their bits: a NaN is above all
            return __uint_as_float(max(__float_as_uint(x), __float_as_uint(y)));
        };
        auto scaled = [](float (&v)[8], float by) {  // returns the sum
            float z = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) z += v[k] *= by;
            return z;
        };
        if constexpr (C::kQReg) {
            uint4 raw[R::kGroups][kRaw];
            float m = 0.f;
#pragma unroll
            for (int g = 0; g < R::kGroups; ++g) load(r, 32 * g + 8 * c, raw[g]);
            if constexpr (F32) {
#pragma unroll
                for (int g = 0; g < R::kGroups; ++g) {
                    float v[8];
                    octet(raw[g], v);
#pragma unroll
                    for (int k = 0; k < 8; ++k) m = larger(m, fabsf(v[k]));
                }
            } else {  // magnitudes as whole numbers, two at a time
                uint32_t m2 = 0;
#pragma unroll
                for (int g = 0; g < R::kGroups; ++g) {
                    const uint32_t w[4] = {raw[g][0].x, raw[g][0].y, raw[g][0].z, raw[g][0].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) m2 = __vmaxu2(m2, w[k] & 0x7fff7fffu);
                }
                m = larger(__uint_as_float(m2 << 16), __uint_as_float(m2 & 0xffff0000u));
            }
            m = larger(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = larger(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const float by = to_f16_range(m, C::kQTo);
            undo(0, __shfl_sync(0xffffffffu, by, 8 * c));  // lane 4 h holds head h
            undo(1, __shfl_sync(0xffffffffu, by, 8 * c + 4));
            // 2^-10 (and 16 times it on the sixteenths) everywhere gives the sums, where the scores
            // will be
            const uint32_t ones[4] = {0x14001400u, 0x14001400u, 0x24002400u, 0x24002400u};
#pragma unroll
            for (int g = 0; g < R::kGroups; ++g) {
                float v[8], d[4] = {0.f, 0.f, 0.f, 0.f};
                octet(raw[g], v);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] *= by;
                split_f16<kQTerms>(qf[g], v);
#pragma unroll
                for (int k = kQTerms - 1; k >= 0; --k) {
                    mma_f16_16816(d, ones, qf[g][k][0], qf[g][k][1]);
                    mma_f16_16816(d, ones, qf[g][k][2], qf[g][k][3]);
                }
                qz[g][0] = d[0] * (C::kUnit * 0x1p10f);
                qz[g][1] = d[1] * (C::kUnit * 0x1p10f);
            }
        } else {
            constexpr int kOcts = R::kPad / 8;
            float *sums = reinterpret_cast<float *>(sQ + kQTerms * kHeads * C::kQRow), *bys = sums + R::kGroups * kHeads;
            for (int h = warp; h < kHeads; h += C::kWarps) {
                float m = 0.f;
                for (int o = lane; o < kOcts; o += 32) {
                    uint4 x[kRaw];
                    float v[8];
                    load(h, 8 * o, x);
                    octet(x, v);
#pragma unroll
                    for (int k = 0; k < 8; ++k) m = larger(m, fabsf(v[k]));
                }
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) m = larger(m, __shfl_xor_sync(0xffffffffu, m, off));
                const float by = to_f16_range(m, C::kQTo);
                for (int o0 = 0; o0 < kOcts; o0 += 32) {
                    const int o = min(o0 + lane, kOcts - 1);  // (a group's four lanes are all there or none)
                    uint4 x[kRaw];
                    float v[8];
                    uint32_t t[kQTerms][4];
                    load(h, 8 * o, x);  // (again, from L1)
                    octet(x, v);
                    float z = scaled(v, by);
                    split_f16<kQTerms>(t, v);
#pragma unroll
                    for (int k = 0; k < kQTerms; ++k)
                        *reinterpret_cast<uint4 *>(sQ + (k * kHeads + h) * C::kQRow + 16 * o) =
                            make_uint4(t[k][0], t[k][1], t[k][2], t[k][3]);
                    z += __shfl_xor_sync(0xffffffffu, z, 1);
                    z += __shfl_xor_sync(0xffffffffu, z, 2);
                    if ((lane & 3) == 0 && o0 + lane < kOcts) sums[o / 4 * kHeads + h] = z * C::kUnit;
                }
                if (lane == 0) bys[h] = by;
            }
            __syncthreads();
            undo(0, bys[2 * c]);
            undo(1, bys[2 * c + 1]);
        }
        fetch_queries(pi + 1, known);
        // one more piece for the table, while the first tile is on its way
        one_more();
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
                {
                    const int row = valid + i / (2 * R::kGroups), off = R::kParamK + 4 * (i % (2 * R::kGroups));
                    *reinterpret_cast<uint32_t *>(tile + row * C::kPitch + C::place(off, (row & 7) << 4)) = 0u;
                }
                __syncwarp();
            }
            // ---- S^T: by groups, each scaled by its keys' scales -----------------------------
            float sc[C::kSub][4];
#pragma unroll
            for (int u = 0; u < C::kSub; ++u) sc[u][0] = sc[u][1] = sc[u][2] = sc[u][3] = 0.f;
#pragma unroll
            for (int st = 0; st < kSets; ++st) {
                uint32_t qs[C::kQReg ? 1 : kSet][kQTerms][4];
                float zs[C::kQReg ? 1 : kSet][2];
                if constexpr (!C::kQReg) {
#pragma unroll
                    for (int j = 0; j < kSet; ++j) {
                        const int g = st * kSet + j;
#pragma unroll
                        for (int k = 0; k < kQTerms; ++k) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(sQ + (k * kHeads + r) * C::kQRow + 16 * (4 * g + c));
                            qs[j][k][0] = v.x, qs[j][k][1] = v.y, qs[j][k][2] = v.z, qs[j][k][3] = v.w;
                        }
                        const float2 z = *reinterpret_cast<const float2 *>(sQ + kQTerms * kHeads * C::kQRow + 4 * (g * kHeads + 2 * c));
                        zs[j][0] = z.x, zs[j][1] = z.y;
                    }
                }
#pragma unroll
                for (int u = 0; u < C::kSub; ++u) {
                    const unsigned char *x = tile + (16 * u + kr) * C::kPitch, *y = x + 8 * C::kPitch;
                    uint32_t wx[kSet], wy[kSet], px[kSet], py[kSet];
                    lds_words<C>(wx, x, 4 * kSet * (4 * st + c), sw_r);
                    lds_words<C>(wy, y, 4 * kSet * (4 * st + c), sw_r);
                    lds_words<C>(px, x, R::kParamK + 4 * kSet * st, sw_r);
                    lds_words<C>(py, y, R::kParamK + 4 * kSet * st, sw_r);
#pragma unroll
                    for (int j = 0; j < kSet; ++j) {
                        const int g = st * kSet + j;
                        const float fx = q4_scale(px[j]), fy = q4_scale(py[j]);
                        const uint32_t ux = wx[j] >> 8, uy = wy[j] >> 8;
                        // 2^-20 (64 + c) and 16 times that, or (F32) c - z and 16 (c - z)
                        constexpr uint32_t kOr = F32 ? 0x64006400u : 0x14001400u;
                        const uint32_t bx[2] = {F32 ? f16_bias(px[j], 0) : 0x13801380u, F32 ? f16_bias(px[j], 4) : 0u};
                        const uint32_t by[2] = {F32 ? f16_bias(py[j], 0) : 0x13801380u, F32 ? f16_bias(py[j], 4) : 0u};
                        const uint32_t a0[4] = {f16_codes<kOr>(wx[j], 0, bx[0]), f16_codes<kOr>(wy[j], 0, by[0]),
                                                f16_codes<kOr>(wx[j], 4, bx[1]), f16_codes<kOr>(wy[j], 4, by[1])};
                        const uint32_t a1[4] = {f16_codes<kOr>(ux, 0, bx[0]), f16_codes<kOr>(uy, 0, by[0]), f16_codes<kOr>(ux, 4, bx[1]),
                                                f16_codes<kOr>(uy, 4, by[1])};
                        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int k = kQTerms - 1; k >= 0; --k) {
                            const uint32_t *q = C::kQReg ? qf[C::kQReg ? g : 0][k] : qs[C::kQReg ? 0 : j][k];
                            mma_f16_16816(d, a0, q[0], q[1]);
                            mma_f16_16816(d, a1, q[2], q[3]);
                        }
                        if constexpr (F32) {  // (the query is large: 2^-24 keeps a large scale from overflowing)
                            sc[u][0] = fmaf(fx, d[0] * C::kUnit, sc[u][0]);
                            sc[u][1] = fmaf(fx, d[1] * C::kUnit, sc[u][1]);
                            sc[u][2] = fmaf(fy, d[2] * C::kUnit, sc[u][2]);
                            sc[u][3] = fmaf(fy, d[3] * C::kUnit, sc[u][3]);
                        } else {
                            const float *z = C::kQReg ? qz[C::kQReg ? g : 0] : zs[C::kQReg ? 0 : j];
                            const float zx = __uint_as_float(px[j] & 0xffff0000u) - 64.f;  // 64 + z
                            const float zy = __uint_as_float(py[j] & 0xffff0000u) - 64.f;
                            sc[u][0] = fmaf(fx, fmaf(-zx, z[0], d[0]), sc[u][0]);
                            sc[u][1] = fmaf(fx, fmaf(-zx, z[1], d[1]), sc[u][1]);
                            sc[u][2] = fmaf(fy, fmaf(-zy, z[0], d[2]), sc[u][2]);
                            sc[u][3] = fmaf(fy, fmaf(-zy, z[1], d[3]), sc[u][3]);
                        }
                    }
                }
            }
            // ---- the log2 domain, the cap, the mask ------------------------------------------
#pragma unroll
            for (int u = 0; u < C::kSub; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[u][e] = sc[u][e] * pre[e & 1] * hs[e & 1];
            if (a.cap_log2 > 0.f) {
#pragma unroll
                for (int u = 0; u < C::kSub; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sc[u][e] = F32 ? a.cap_log2 * tanhf(sc[u][e] * a.over_cap_log2)
                                       : capped_score_close(sc[u][e] * a.over_cap_log2, a.cap_log2);
            }
            if (valid < C::kKeys) {
#pragma unroll
                for (int u = 0; u < C::kSub; ++u) {
                    if (16 * u + kr >= valid) sc[u][0] = sc[u][1] = -INFINITY;
                    if (16 * u + 8 + kr >= valid) sc[u][2] = sc[u][3] = -INFINITY;
                }
            }
            // ---- running reference and sum.  Any reference within 2^8 of the maximum serves; it
            // moves (to the maximum) only when some score has outgrown it, which a vote tells --
            float t[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                t[e] = fmaxf(sc[0][e], sc[0][e + 2]);
#pragma unroll
                for (int u = 1; u < C::kSub; ++u) t[e] = fmaxf(t[e], fmaxf(sc[u][e], sc[u][e + 2]));
            }
            if (__any_sync(0xffffffffu, t[0] > m_ref[0] + kRescaleBy || t[1] > m_ref[1] + kRescaleBy)) {
                float corr[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    t[e] = fmaxf(t[e], __shfl_xor_sync(0xffffffffu, t[e], 4));
                    t[e] = fmaxf(t[e], __shfl_xor_sync(0xffffffffu, t[e], 8));
                    t[e] = fmaxf(t[e], __shfl_xor_sync(0xffffffffu, t[e], 16));
                    const float m_new = fmaxf(m_ref[e], t[e]);
                    corr[e] = m_new == -INFINITY ? 1.f : fast_exp2(m_ref[e] - m_new);
                    l_run[e] *= corr[e];
                    m_ref[e] = m_new;
                }
#pragma unroll
                for (int i = 0; i < C::kMt; ++i) {
                    acc[i][0] *= corr[0];
                    acc[i][1] *= corr[1];
                    acc[i][2] *= corr[0];
                    acc[i][3] *= corr[1];
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float m_use = m_ref[e] == -INFINITY ? 0.f : m_ref[e];
#pragma unroll
                for (int u = 0; u < C::kSub; ++u) {
                    sc[u][e] = fast_exp2(sc[u][e] - m_use);
                    sc[u][e + 2] = fast_exp2(sc[u][e + 2] - m_use);
                    l_run[e] += sc[u][e] + sc[u][e + 2];
                }
            }
            // ---- O^T += V^T (P s)^T ----------------------------------------------------------
#pragma unroll
            for (int st = 0; st < kSets; ++st) {
#pragma unroll
                for (int u = 0; u < C::kSub; ++u) {
                    const unsigned char *rows = tile + 16 * u * C::kPitch;
                    const unsigned char *x = rows + kr * C::kPitch, *y = x + 8 * C::kPitch;
                    const unsigned char *k0p = rows + kp * C::kPitch, *k1p = k0p + 2 * C::kPitch;
                    uint32_t px[kSet], py[kSet], q0[kSet], q1[kSet], q2[kSet], q3[kSet], ab[kSet], cd[kSet];
                    lds_words<C>(px, x, R::kParamV + 4 * kSet * st, sw_r);
                    lds_words<C>(py, y, R::kParamV + 4 * kSet * st, sw_r);
                    lds_words<C>(q0, k0p, R::kParamV + 4 * kSet * st, sw_0);
                    lds_words<C>(q1, k1p, R::kParamV + 4 * kSet * st, sw_1);
                    lds_words<C>(q2, k0p + 8 * C::kPitch, R::kParamV + 4 * kSet * st, sw_0);
                    lds_words<C>(q3, k1p + 8 * C::kPitch, R::kParamV + 4 * kSet * st, sw_1);
                    const int vo = R::kV + 2 * kSet * (8 * st + r);
                    v_pairs<C>(ab, k0p, k1p, vo, sw_0, sw_1);
                    v_pairs<C>(cd, k0p + 8 * C::kPitch, k1p + 8 * C::kPitch, vo, sw_0, sw_1);
#pragma unroll
                    for (int j = 0; j < kSet; ++j) {
                        const int g = st * kSet + j;
                        const float fx = q4_scale(px[j]), fy = q4_scale(py[j]);
                        uint32_t w0[kTerms], w1[kTerms];
                        if constexpr (Twin) {
                            w0[0] = term2(sc[u][0] * fx, sc[u][1] * fx, twin_by);
                            w1[0] = term2(sc[u][2] * fy, sc[u][3] * fy, twin_by);
                        } else {
                            split2<kTerms>(w0, sc[u][0] * fx, sc[u][1] * fx);
                            split2<kTerms>(w1, sc[u][2] * fy, sc[u][3] * fy);
                        }
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
        // this warp's share of heads 2 c and 2 c + 1: 2^(m - M) / sum over the warps of l 2^(m - M)
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
            f[e] = l == 0.f ? 0.f : fast_exp2(m_ref[e] - base) / l;
            if (warp == 0 && r == 0 && 2 * c + e < g_cnt) {
                const int64_t bh = (int64_t)p.b * a.n_heads + h_base + 2 * c + e;
                const float lse2 = M + log2f(l);
                if (a.defer_join && p.slot == 0) a.piece_count[bh] = p.nseg;
                if (!single) a.part_lse[bh * a.max_splits + p.slot] = lse2;
                else if (a.lse != nullptr) a.lse[bh] = lse2 * kLn2;
            }
        }
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
            for (int v = tid; v < (Twin ? kTwinHeads : kHeads) * kV4; v += C::kThreads) {
                const int h = v / kV4, x = 4 * (v % kV4), d = 16 * i0 + x;
                if (h >= g_cnt || d >= D) continue;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < C::kWarps; ++w) {
                    for (int col = h; col < (Twin ? kHeads : h + 1); col += kTwinHeads) {
                        const float4 t = *reinterpret_cast<const float4 *>(park + (w * kHeads + col) * C::kParkPitch + x);
                        o.x += t.x; o.y += t.y; o.z += t.z; o.w += t.w;
                    }
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
            joins[n_joins++] = Join{p.b, h_base, g_cnt, p.nseg, (p.b * a.n_kv_heads + p.hk) * HB + p.hb, 0};
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
    if (a.defer_join) return;
    // ---- the units whose last piece was this CTA's: weights 2^{lse_c - lse} over their pieces ----
    __syncthreads();  // every thread's partials are written
    if (*abort_flag) return;
    // (each thread's partials happen before the barrier, that before the ticket's release; a last
    // ticket's acquire before the next barrier, that before the reads, which skip L1)
    if (lane == 0 && warp < 2 && joins[warp].nseg > 0)  // a ticket a warp: they take a round trip each
        joins[warp].last = add_acq_rel(a.counters + joins[warp].unit, 1) == joins[warp].nseg - 1;
    __syncthreads();
    for (int k = 0; k < 2; ++k) {
        const Join j = joins[k];
        if (!j.last) continue;
        for (int v = tid; v < j.g_cnt * (D / 4); v += C::kThreads) {
            const int h = j.h_base + v / (D / 4), d = 4 * (v % (D / 4));
            const int64_t bh = (int64_t)j.b * a.n_heads + h;
            const float *pl = a.part_lse + bh * a.max_splits;
            const float *po = a.part_o + bh * a.max_splits * D + d;
            float m = -INFINITY, z = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            constexpr int kAhead = 8;  // pieces in flight
            for (int s0 = 0; s0 < j.nseg; s0 += kAhead) {
                float l[kAhead], mn = m;
                float4 w[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const bool there = s0 + i < j.nseg;
                    l[i] = there ? __ldcg(pl + s0 + i) : -INFINITY;
                    w[i] = there ? __ldcg(reinterpret_cast<const float4 *>(po + (int64_t)(s0 + i) * D))
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
                for (int i = 0; i < kAhead; ++i) mn = fmaxf(mn, l[i]);
                const float base = mn == -INFINITY ? 0.f : mn, cf = fast_exp2(m - base);
                z *= cf; o.x *= cf; o.y *= cf; o.z *= cf; o.w *= cf;
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const float e = fast_exp2(l[i] - base);
                    z += e;
                    o.x = fmaf(e, w[i].x, o.x); o.y = fmaf(e, w[i].y, o.y);
                    o.z = fmaf(e, w[i].z, o.z); o.w = fmaf(e, w[i].w, o.w);
                }
                m = mn;
            }
            const float rz = z == 0.f ? 0.f : 1.f / z;
            T *dst = static_cast<T *>(a.out) + (int64_t)j.b * a.out_rs + (int64_t)h * D + d;
            if constexpr (F32)
                *reinterpret_cast<float4 *>(dst) = make_float4(o.x * rz, o.y * rz, o.z * rz, o.w * rz);
            else
                *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(o.x * rz, o.y * rz), pack_bf16x2(o.z * rz, o.w * rz));
            if (d == 0 && a.lse != nullptr) a.lse[bh] = (m + log2f(z)) * kLn2;
        }
        if (tid == 0) a.counters[j.unit] = 0;  // ready for the next call
    }
}

template <int D, bool F32, bool Wide, bool Twin>
cudaError_t launch_q4_d(const Q4DecodeArgs &a, int grid, cudaStream_t s) {
    using C = Q4Cfg<D, F32, Wide, Twin>;
    cudaError_t e = cudaFuncSetAttribute(decode_q4_kernel<D, F32, Wide, Twin>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    decode_q4_kernel<D, F32, Wide, Twin><<<grid, C::kThreads, C::kSmem, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess || !a.defer_join) return e;
    const JoinArgs j{a.part_o, a.part_lse, a.piece_count, a.max_splits, a.n_heads, a.out, a.out_rs, a.lse};
    return launch_split_join<D, F32>(j, (int64_t)a.batch * a.n_heads, s);
}

// Keys per CTA, were all units as long as they may be, from which the wide form is taken.  At 3449
// 32 ragged sequences take 30.7 us wide and 28.6 narrow, 8 equally long ones 41.5 and 41.4; at
// 6898 47.4 and 45.2, 71.0 and 73.4; at 13797 83.4 and 83.1, 131 and 136.
constexpr int64_t kWideKeys = 6144;

template <int D, bool F32, bool Wide, bool Twin>
int occupancy_of() {
    using C = Q4Cfg<D, F32, Wide, Twin>;
    static Occupancy occupancy;
    return occupancy(decode_q4_kernel<D, F32, Wide, Twin>, C::kThreads, C::kSmem);
}

// grid, wide, box_rows, and the keys of a tile, for `units` units of up to `keys` keys
template <int D, bool F32, bool Twin>
int shape_of(Q4Plan *p, int sms, int64_t units, int64_t keys) {
    using C = Q4Cfg<D, F32, false, Twin>;
    p->wide = 0;
    p->twin = Twin;
    if constexpr (kHasWide<D, F32>) {
        using W = Q4Cfg<D, F32, true, Twin>;
        p->grid = sms * occupancy_of<D, F32, true, Twin>();
        if (p->grid > 0 && units * keys / p->grid >= kWideKeys) {
            p->wide = 1;
            p->box_rows = W::kKeys;
            return W::kTileKeys;
        }
    }
    p->grid = sms * occupancy_of<D, F32, false, Twin>();
    p->box_rows = C::kKeys;
    return C::kTileKeys;
}

// calls f<D, F32, Twin> for a supported head_dim and type (fp32 queries need their columns)
#define LAT_Q4_CASE(D, bf16, twin, f, ...) \
    case D: return !(bf16) ? f<D, true, false>(__VA_ARGS__) : (twin) ? f<D, false, true>(__VA_ARGS__) : f<D, false, false>(__VA_ARGS__);
#define LAT_Q4_DISPATCH(head_dim, bf16, twin, f, other, ...) \
    switch (head_dim) {                                      \
        LAT_Q4_CASE(64, bf16, twin, f, __VA_ARGS__)          \
        LAT_Q4_CASE(80, bf16, twin, f, __VA_ARGS__)          \
        LAT_Q4_CASE(128, bf16, twin, f, __VA_ARGS__)         \
        LAT_Q4_CASE(256, bf16, twin, f, __VA_ARGS__)         \
        LAT_Q4_CASE(512, bf16, twin, f, __VA_ARGS__)         \
        default: return other;                               \
    }
int shape(int head_dim, bool bf16, bool twin, Q4Plan *p, int sms, int64_t units, int64_t keys) {
    LAT_Q4_DISPATCH(head_dim, bf16, twin, shape_of, 0, p, sms, units, keys)
}
template <int D, bool F32, bool Twin>
cudaError_t launch_q4(const Q4DecodeArgs &a, int grid, bool wide, cudaStream_t s) {
    if constexpr (kHasWide<D, F32>)
        if (wide) return launch_q4_d<D, F32, true, Twin>(a, grid, s);
    return launch_q4_d<D, F32, false, Twin>(a, grid, s);
}

}  // namespace

bool plan_decode_q4(int batch, int n_heads, int n_kv_heads, int head_dim, bool bf16, int max_kv_len, int num_sms,
                    Q4Plan *p) {
    const int G = n_heads / n_kv_heads, HB = (G + kHeads - 1) / kHeads;
    const int64_t units = (int64_t)batch * n_kv_heads * HB;
    // join grid: one CTA per (sequence, query head, up to 128 channels)
    if ((int64_t)batch * n_heads * ((head_dim + 127) / 128) > 0x7fffffffLL) return false;
    const int tile = shape(head_dim, bf16, G <= kTwinHeads, p, num_sms, units, max_kv_len);
    if (tile == 0) return false;
    // A unit of n tiles falls into at most n / min_tiles + 2 pieces.  min_tiles keeps that count
    // near 64 or, with few units, near the number of CTAs that each unit must feed.
    const int64_t range = ((int64_t)std::max(max_kv_len, 1) + tile - 1) / tile;
    if (units * (range + kUnitCost) > 0x7fffffffLL) return false;
    const int64_t target = std::max<int64_t>(64, (p->grid + std::max<int64_t>(units, 1) - 1) / std::max<int64_t>(units, 1));
    p->min_tiles = (int)std::max<int64_t>(1, (range + target - 1) / target);
    // Units of up to two tiles, no more than the CTAs: one each, and nothing to join (8 KV heads,
    // head_dim 64: one sequence of 512 keys 7.3 instead of 8.0 us, 32 ragged ones of up to 512 8.6
    // instead of 10.2; with three tiles it gains nothing).
    p->whole = range <= 2 && units <= p->grid;
    if (p->whole) p->min_tiles = (int)range + kUnitCost;
    p->max_splits = (int)((range + p->min_tiles - 1) / p->min_tiles) + 2;
    // With few units, cut finely, the CTA that joins one would read tens of partials after its
    // stream; a second kernel takes them then.
    p->defer_join = units * 8 < p->grid && p->max_splits > 16;
    auto round256 = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t rows = (size_t)batch * n_heads;
    p->part_o_bytes = round256(rows * p->max_splits * head_dim * 4);
    p->part_lse_bytes = round256(rows * p->max_splits * 4);
    // pieces per (sequence, head), or tickets per unit
    p->total_bytes = p->part_o_bytes + p->part_lse_bytes + round256((p->defer_join ? rows : (size_t)units) * 4);
    return true;
}

cudaError_t launch_decode_q4(const Q4DecodeArgs &a, bool bf16, const Q4Plan &p, cudaStream_t s) {
    LAT_Q4_DISPATCH(a.head_dim, bf16, p.twin != 0, launch_q4, cudaErrorInvalidValue, a, p.grid, p.wide != 0, s)
}

}  // namespace lat
