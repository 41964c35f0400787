// Split-KV decode over 4-bit pools (row layout: fp4.cuh).
//
// The method is decode.cu's: persistent CTAs over equal ranges of the batch's
// work list, online softmax, one partial (O, lse) per range and row, merged by
// the log-sum-exp combine.  What differs:
//   - The list counts units of 16 keys that start at multiples of 16 in their
//     sequence, so that a unit never straddles two 16-token pages: its rows are
//     one contiguous run of the pool when a row is one head group, and a unit
//     is two bulk copies (K, V) instead of 32; with more groups it is two
//     tensor-map boxes of 16 rows (21 sequences, 103,000 keys, 16 heads of 128:
//     56 us, by rows 88).
//   - A CTA takes one head group (gs KV heads, one consumer warp each).
//   - The codes are widened in registers: E2M1 to f16 by the hardware
//     conversion, times the block's E4M3 scale (exact in f16, fp4.cuh), and
//     both contractions run in f16 with fp32 accumulation.  The head's K scale
//     is a factor of the score, its V scale one of the output, so neither q
//     (bf16 values in f16's range are exact) nor K nor V is rounded; only P is.
//
// Fragments of mma.sync m16n8k16 (r8 = lane / 4, q4 = lane % 4).  The order of
// the contracted index and of the rows is free, so each lane takes what lies
// together in the row:
//   S (16 keys x 8 heads) = K Q^T: lane q4 takes elements [D/4 q4, D/4 q4 + D/4)
//     of its two keys: one 16-byte load per key (8 at D = 64) and two scales.
//   O^T (D x 8 heads) += V^T P^T: lane r8 takes elements [D/8 r8, + D/8) of its
//     four keys: one 8-byte load (4) and one scale per key; the words of two
//     keys are interleaved nibble by nibble, so that a byte holds one element
//     of both and converts to the pair the fragment wants.
//   P goes from the score's layout to the second product's with movmatrix.
// Row r of the score fragment is key r ^ ((r >> 1) & 1): with rows 64 bytes
// apart modulo the banks' 128 this halves the conflicts of the V loads.
//
// The running maximum is lazy as in decode.cu; here a vote decides whether any
// score exceeds it by more than 2^8, so that the usual unit needs no shuffle.
//
// What bounds it: HBM delivers a unit of a head (2304 bytes at D = 128) every 98
// clocks per SM, its consumer warps need about 300 instructions for it and issue
// 2.5 per clock (64 conversions, 64 multiplies, 16 MMAs, the rest of the softmax
// and addresses).  256 log-uniform contexts up to 32768 (2.38 GB): 423 us, 5.6
// TB/s, 0.83 of the measured copy bandwidth; one unit at a time 428 us, with
// 64-bit walks and six more live registers 448 (more spills), 472 before the
// pairs.  As built <128, 8> has 96 registers, for two CTAs an SM, and spills 80
// bytes a thread.
// At D = 64 half the bytes come with more than half the instructions: 64
// sequences of up to 4096 keys 24 us, 0.40.  One sequence of 20011 keys takes 14.8
// us: ranges sized by SMs fill half of the CTA slots.
#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

#include "decode_impl.cuh"
#include "fp4.cuh"
#include "pa_device.cuh"
#include "pa_internal.h"
#include "pdl.cuh"
#include "tensor_map.cuh"

namespace pa {

PA_ERROR_WORD_ACCESSOR(error_word_decode_fp4)

namespace {

constexpr int kUnit = 16;         // keys of a unit

struct Fp4DecodeArgs {
    const __nv_bfloat16 *q;
    const uint8_t *k_cache;
    const uint8_t *v_cache;
    const int32_t *page_table;
    int64_t pt_stride;
    const int32_t *cache_seqlens;
    int32_t num_seqs;
    int32_t num_q_heads;
    int32_t group;                // query heads per KV head
    int32_t page_size;
    int64_t num_pages;
    float scale_log2;
    int32_t min_units;            // smallest range, in units
    int32_t max_seqlen_k;
    int32_t max_splits;
    int32_t head_groups;
    int32_t row_bytes;
    float *o_part;
    float *lse_part;
    const float *k_scale;
    const float *v_scale;
    int32_t window;
    int32_t overlap_previous;     // do not wait for the kernel before
    int32_t *ws_header;           // [0] = T, in units
    int32_t *ws_prefix;           // [B+1] exclusive prefix of the sequences' units
};

// Page size 16 and more than one head group (BOX): the pools as rows of 32-bit
// words.  An instantiation of its own: the boxes in the code of all calls cost
// 256 contexts up to 32768 keys 445 us instead of 423.
struct Fp4Maps {
    CUtensorMap k, v;
};
struct Fp4NoMaps {};
template <bool BOX>
using Fp4MapsOf = std::conditional_t<BOX, Fp4Maps, Fp4NoMaps>;

template <int D, int HPC>
struct Fp4Smem {
    static constexpr int kCodes = HPC * D / 2;
    static constexpr int kRow = (kCodes + HPC * D / 16 + 15) / 16 * 16;    // a key's group: codes, scales, padding
    static constexpr int kStage = 2 * kUnit * kRow;                        // K rows, then V rows
    // Ring: about 160 KiB per SM over the CTAs that fit (kCtas below).
    static constexpr int kCtas = HPC == 8 ? 2 : HPC == 4 ? 3 : HPC == 2 ? 6 : 9;
    static constexpr int kFit = 184320 / kCtas / kStage;
    static constexpr int kStages = kFit > 8 ? 8 : kFit;
    static constexpr int kRing = kStages * kStage;
    static_assert(kStages >= 4, "ring too short");
};

// First key and number of keys of sequence b that its query sees.
__device__ __forceinline__ int seq_keys(const Fp4DecodeArgs &a, int b, int &lo) {
    int L = a.cache_seqlens[b];
    L = L < 0 ? 0 : (L > a.max_seqlen_k ? a.max_seqlen_k : L);
    lo = (a.window > 0 && L > a.window) ? L - a.window : 0;
    return L;
}

// Exclusive prefix of the sequences' units into prefix[0 .. B] (all threads).
__device__ __forceinline__ void fp4_prefix(const Fp4DecodeArgs &a, int32_t *prefix) {
    const int B = a.num_seqs;
    for (int b = threadIdx.x; b < B; b += blockDim.x) {
        const int given = a.cache_seqlens[b];
        if (given < 0 || given > a.max_seqlen_k) raise_error(PA_DEVERR_SEQLENS);
        int lo;
        const int L = seq_keys(a, b, lo);
        prefix[b + 1] = L > 0 ? (L - 1) / kUnit - lo / kUnit + 1 : 0;
    }
    if (threadIdx.x == 0) prefix[0] = 0;
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const int per = (B + 31) / 32;
        const int from = 1 + lane * per, to = min(B, lane * per + per);
        int run = 0;
        for (int i = from; i <= to; ++i) run += prefix[i];
        int incl = run;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        int acc = incl - run;
        for (int i = from; i <= to; ++i) {
            acc += prefix[i];
            prefix[i] = acc;
        }
    }
    __syncthreads();
}

// SegmentWalk (decode_impl.cuh) over the list of units, in 32 bits: the call
// has fewer than 2^31 keys over all head groups, so fewer units.
struct UnitWalk {
    const int32_t *pb;
    int B, HG, T, g, g1;
    __device__ __forceinline__ bool next(int &b, int &hg, int &u0, int &u1, int &split, int &span) {
        if (g >= g1) return false;
        int lo = 0, hi = B;           // HG * pb[lo] <= g < HG * pb[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (HG * pb[mid] <= g) lo = mid; else hi = mid;
        }
        b = lo;
        const int U = pb[b + 1] - pb[b];                  // > 0 by the invariant
        const int local = g - HG * pb[b];
        hg = local / U;
        u0 = local - hg * U;
        u1 = min(u0 + (g1 - g), U);
        const int first = g / T;
        split = first - (g - u0) / T;
        span = (g + (u1 - u0) - 1) / T - first + 1;
        g += u1 - u0;
        return true;
    }
};

// A box of 16 rows of one head group; x in 32-bit words (a multiple of 4).
__device__ __forceinline__ void tma_load_rows(void *dst, const CUtensorMap *map, int x, int row, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(smem_u32(dst)), "l"(map), "r"(x), "r"(row), "r"(smem_u32(bar)) : "memory");
}

// The producer warp: units [g0, g1) of the list into the ring.
template <int D, int HPC, bool BOX>
__device__ void fp4_produce(const Fp4DecodeArgs &a, const Fp4MapsOf<BOX> &maps, const int32_t *prefix, int T, int g0, int g1,
                            uint8_t *ring, uint64_t *full, uint64_t *empty, int lane) {
    using S = Fp4Smem<D, HPC>;
    const bool paged = a.page_size == 16;
    const bool run = !BOX && paged;                  // one head group: a unit is one contiguous run of rows
    int ctr = 0;
    UnitWalk walk{prefix, a.num_seqs, a.head_groups, T, g0, g1};
    int b, hg, u0, u1, split, span;
    while (walk.next(b, hg, u0, u1, split, span)) {
        const int32_t *pt = a.page_table + (int64_t)b * a.pt_stride;
        int lo;
        const int L = seq_keys(a, b, lo);
        const int first = lo / kUnit;                // the sequence's unit 0
        // Page size 16: lane i holds the page of unit c0 + i, the next 32 are
        // read while these are copied.  Page size 1: lane i the slot of key i
        // of the unit, read one unit ahead.
        auto ids = [&](int u) {
            if (paged) return u + lane < u1 ? pt[first + u + lane] : 0;
            const int j = (first + u) * kUnit + (lane & 15);
            return u < u1 && j >= lo && j < L ? pt[j] : 0;
        };
        int now = 0, ahead = ids(u0);
        for (int u = u0; u < u1; ++u, ++ctr) {
            const int i = paged ? (u - u0) & 31 : 0;
            if (i == 0) {
                now = ahead;
                ahead = ids(u + (paged ? 32 : 1));
            }
            const int key = (first + u) * kUnit;
            const int n0 = max(lo - key, 0), n1 = min(L - key, kUnit);   // keys of the unit that are seen
            const int slot = ctr % S::kStages, round = ctr / S::kStages;
            if (round > 0 && !mbar_wait(&empty[slot], (round - 1) & 1)) return;
            if (lane == 0) mbar_arrive_expect_tx(&full[slot], 2u * (BOX ? kUnit : n1 - n0) * S::kRow);   // a box is loaded whole
            __syncwarp();
            int64_t page = __shfl_sync(0xffffffffu, now, paged ? i : (lane & 15));
            const int tok = lane & 15;
            const bool mine = BOX || run ? (lane & 15) == 0 : (tok >= n0 && tok < n1);
            if (mine) {
                if (page < 0 || page >= a.num_pages) {           // never read outside the pool
                    raise_error(PA_DEVERR_PAGE_RANGE);
                    page = 0;
                }
                if constexpr (BOX) {
                    tma_load_rows(ring + slot * S::kStage + (lane >> 4) * (kUnit * S::kRow), lane < 16 ? &maps.k : &maps.v,
                                  hg * (S::kRow / 4), (int)page * 16, &full[slot]);
                    continue;
                }
                const int at = run ? n0 : tok;
                const int64_t row = paged ? page * 16 + at : page;
                uint8_t *dst = ring + slot * S::kStage + (lane >> 4) * (kUnit * S::kRow) + at * S::kRow;
                const uint8_t *src = (lane < 16 ? a.k_cache : a.v_cache) + row * a.row_bytes + (int64_t)hg * S::kRow;
                bulk_g2s(dst, src, (run ? n1 - n0 : 1) * S::kRow, &full[slot]);
            }
        }
    }
}

__device__ __forceinline__ uint32_t f16x2_of(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// mma_f16_16816 into a fresh accumulator (no registers to clear first).
__device__ __forceinline__ void mma_f16_16816_zero(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Where a consumer lane finds its part of a stage (bytes from its start).
template <int D, int HPC>
struct Fp4Lane {
    using S = Fp4Smem<D, HPC>;
    int k_off, ks_off;            // codes and scales of key place(r8); those of key + 8 are 8 rows on
    int v_off, vs_off;            // codes and scale of key place(2 q4)
    int v_next;                   // from there to key place(2 q4 + 1)
    static __device__ __forceinline__ int place(int r) { return r ^ ((r >> 1) & 1); }   // fragment row -> key of the unit
    __device__ __forceinline__ Fp4Lane(int hw, int lane) {
        const int r8 = lane >> 2, q4 = lane & 3;
        k_off = place(r8) * S::kRow + hw * (D / 2) + q4 * (D / 8);
        ks_off = place(r8) * S::kRow + S::kCodes + hw * (D / 16) + q4 * (D / 64);
        const int v = (kUnit + place(2 * q4)) * S::kRow;
        v_off = v + hw * (D / 2) + r8 * (D / 16);
        vs_off = v + S::kCodes + hw * (D / 16) + (D == 128 ? r8 : r8 >> 1);
        v_next = (place(2 * q4 + 1) - place(2 * q4)) * S::kRow;
    }
};

// Raw scores of a unit: x[0], x[1] of key place(r8) and heads 2 q4, 2 q4 + 1;
// x[2], x[3] of the key 8 on.  Keys outside [n0, n1) give -inf.
template <int D, int HPC>
__device__ __forceinline__ void fp4_scores(const Fp4Lane<D, HPC> &ln, const uint8_t *st, const uint32_t (&qb)[D / 16][2],
                                           int n0, int n1, float *x) {
    using S = Fp4Smem<D, HPC>;
    constexpr int KW = D / 32;                       // words of a lane's part of a row
    float sc[4], sd[4];
    uint32_t kw[2][KW], ks[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint8_t *p = st + 8 * i * S::kRow;
        if constexpr (KW == 4) {
            const uint4 w = *reinterpret_cast<const uint4 *>(p + ln.k_off);
            kw[i][0] = w.x; kw[i][1] = w.y; kw[i][2] = w.z; kw[i][3] = w.w;
            ks[i] = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(p + ln.ks_off));
        } else {
            const uint2 w = *reinterpret_cast<const uint2 *>(p + ln.k_off);
            kw[i][0] = w.x; kw[i][1] = w.y;
            ks[i] = e4m3x2_to_f16x2(p[ln.ks_off]);
        }
    }
#pragma unroll
    for (int w = 0; w < KW; ++w) {                   // a word is two k-steps
        uint32_t a[4], b[4];
        e2m1x8_to_f16x8(kw[0][w], a);
        e2m1x8_to_f16x8(kw[1][w], b);
        const uint32_t s0 = w < 2 ? f16_dup_lo(ks[0]) : f16_dup_hi(ks[0]);
        const uint32_t s1 = w < 2 ? f16_dup_lo(ks[1]) : f16_dup_hi(ks[1]);
        const uint32_t fa[4] = {hmul2_bits(a[0], s0), hmul2_bits(b[0], s1), hmul2_bits(a[1], s0), hmul2_bits(b[1], s1)};
        const uint32_t fb[4] = {hmul2_bits(a[2], s0), hmul2_bits(b[2], s1), hmul2_bits(a[3], s0), hmul2_bits(b[3], s1)};
        if (w == 0) {
            mma_f16_16816_zero(sc, fa, qb[0][0], qb[0][1]);
            mma_f16_16816_zero(sd, fb, qb[1][0], qb[1][1]);
        } else {
            mma_f16_16816(sc, fa, qb[2 * w][0], qb[2 * w][1]);
            mma_f16_16816(sd, fb, qb[2 * w + 1][0], qb[2 * w + 1][1]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = sc[i] + sd[i];
    if (n0 > 0 || n1 < kUnit) {
        const int tk = Fp4Lane<D, HPC>::place((threadIdx.x & 31) >> 2);
        const bool s0 = tk >= n0 && tk < n1, s1 = tk + 8 >= n0 && tk + 8 < n1;
        x[0] = s0 ? x[0] : -INFINITY;
        x[1] = s0 ? x[1] : -INFINITY;
        x[2] = s1 ? x[2] : -INFINITY;
        x[3] = s1 ? x[3] : -INFINITY;
    }
}

// oacc += V^T P^T of a unit, P the weights of fp4_scores' places.
template <int D, int HPC>
__device__ __forceinline__ void fp4_values(const Fp4Lane<D, HPC> &ln, const uint8_t *st, const float *p, int n0, int n1,
                                           float (&oacc)[D / 16][4]) {
    using S = Fp4Smem<D, HPC>;
    constexpr int VW = D / 64;                       // words of a lane's part of a row
    uint32_t vw[4][VW], vs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint8_t *q = st + 8 * (i >> 1) * S::kRow;
        const int off = ln.v_off + ((i & 1) ? ln.v_next : 0);
        if constexpr (VW == 2) {
            const uint2 w = *reinterpret_cast<const uint2 *>(q + off);
            vw[i][0] = w.x; vw[i][1] = w.y;
        } else {
            vw[i][0] = *reinterpret_cast<const uint32_t *>(q + off);
        }
        vs[i] = q[ln.vs_off + ((i & 1) ? ln.v_next : 0)];
    }
    if (n0 > 0 || n1 < kUnit) {                      // keys that are not seen may hold anything: a zero scale clears them
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = Fp4Lane<D, HPC>::place(2 * (threadIdx.x & 3) + (i & 1)) + 8 * (i >> 1);
            if (t < n0 || t >= n1) vs[i] = 0u;
        }
    }
    const uint32_t pb0 = movmatrix_trans(f16x2_of(p[0], p[1]));
    const uint32_t pb1 = movmatrix_trans(f16x2_of(p[2], p[3]));
    const uint32_t sa = e4m3x2_to_f16x2(vs[0] | (vs[1] << 8)), sb = e4m3x2_to_f16x2(vs[2] | (vs[3] << 8));
#pragma unroll
    for (int w = 0; w < VW; ++w) {
        constexpr uint32_t m = 0x0f0f0f0fu;
        // even elements of both keys in one word, odd ones in another
        uint32_t ea[4], oa[4], eb[4], ob[4];
        e2m1x8_to_f16x8((vw[0][w] & m) | ((vw[1][w] << 4) & ~m), ea);
        e2m1x8_to_f16x8(((vw[0][w] >> 4) & m) | (vw[1][w] & ~m), oa);
        e2m1x8_to_f16x8((vw[2][w] & m) | ((vw[3][w] << 4) & ~m), eb);
        e2m1x8_to_f16x8(((vw[2][w] >> 4) & m) | (vw[3][w] & ~m), ob);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t f[4] = {hmul2_bits(ea[i], sa), hmul2_bits(oa[i], sa), hmul2_bits(eb[i], sb), hmul2_bits(ob[i], sb)};
            mma_f16_16816(oacc[4 * w + i], f, pb0, pb1);
        }
    }
}

// Consumer warp hw: KV head hg * HPC + hw of each segment of the same range.
// Units are taken in pairs: one vote and one maximum for 32 keys, and two
// independent score chains in flight.
template <int D, int HPC>
__device__ void fp4_consume(const Fp4DecodeArgs &a, const int32_t *prefix, int T, int g0, int g1,
                            const uint8_t *ring, uint64_t *full, uint64_t *empty, int hw, int lane) {
    using S = Fp4Smem<D, HPC>;
    constexpr int KS = D / 16;                       // k-steps of the score = tiles of O
    const int r8 = lane >> 2, q4 = lane & 3;
    const int G = a.group;
    const Fp4Lane<D, HPC> ln(hw, lane);
    int slot = 0;
    uint32_t phase = 0;
    UnitWalk walk{prefix, a.num_seqs, a.head_groups, T, g0, g1};
    int b, hg, u0, u1, split, span;
    while (walk.next(b, hg, u0, u1, split, span)) {
        const int kvh = hg * HPC + hw;
        const int h0 = kvh * G;
        int lo;
        const int L = seq_keys(a, b, lo);
        const int first = lo / kUnit;
        const float sl2 = fp4_score_scale(a.scale_log2, a.k_scale[kvh]);     // raw score -> log2 units
        const float lazy = kLazyRescale / sl2;
        uint32_t qb[KS][2];
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) qb[kk][0] = qb[kk][1] = 0u;
        if (r8 < G) {
            const uint2 *qrow = reinterpret_cast<const uint2 *>(a.q + ((int64_t)b * a.num_q_heads + h0 + r8) * D + q4 * (D / 4));
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) {
                const uint2 w = qrow[kk];
                qb[kk][0] = f16x2_of(bf16lo(w.x), bf16hi(w.x));
                qb[kk][1] = f16x2_of(bf16lo(w.y), bf16hi(w.y));
            }
        }
        float oacc[KS][4];
#pragma unroll
        for (int mt = 0; mt < KS; ++mt) oacc[mt][0] = oacc[mt][1] = oacc[mt][2] = oacc[mt][3] = 0.f;
        // the running maximum in log2 units, the raw score beyond which it moves
        float m_run[2] = {-INFINITY, -INFINITY}, limit[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
        for (int u = u0; u < u1; u += 2) {
            const bool two = u + 1 < u1;
            const int key = (first + u) * kUnit;
            const int na = lo - key, nb = L - key;   // keys na .. nb - 1 from the first unit's start are seen
            const uint8_t *sta = ring + slot * S::kStage;
            uint64_t *ea = &empty[slot], *eb = nullptr;
            if (!mbar_wait(&full[slot], phase)) return;
            __syncwarp();
            if (++slot == S::kStages) { slot = 0; phase ^= 1u; }
            float x[8];
            fp4_scores<D, HPC>(ln, sta, qb, na, nb, x);
            const uint8_t *stb = ring + slot * S::kStage;
            if (two) {
                eb = &empty[slot];
                if (!mbar_wait(&full[slot], phase)) return;
                __syncwarp();
                if (++slot == S::kStages) { slot = 0; phase ^= 1u; }
                fp4_scores<D, HPC>(ln, stb, qb, na - kUnit, nb - kUnit, x + 4);
            } else {
                x[4] = x[5] = x[6] = x[7] = -INFINITY;
            }
            // ---- online softmax in the log2 domain
            float top[2] = {fmaxf(fmaxf(x[0], x[2]), fmaxf(x[4], x[6])), fmaxf(fmaxf(x[1], x[3]), fmaxf(x[5], x[7]))};
            if (__any_sync(0xffffffffu, top[0] > limit[0] || top[1] > limit[1])) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float mx = top[j];
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    if (mx > limit[j]) {
                        const float alpha = fast_exp2(m_run[j] - mx * sl2);      // 0 when m_run = -inf
                        l_run[j] *= alpha;
#pragma unroll
                        for (int mt = 0; mt < KS; ++mt) {
                            oacc[mt][j] *= alpha;
                            oacc[mt][2 + j] *= alpha;
                        }
                        m_run[j] = mx * sl2;
                        limit[j] = mx + lazy;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = fast_exp2(fmaf(x[i], sl2, -m_run[i & 1]));
            l_run[0] += (x[0] + x[2]) + (x[4] + x[6]);
            l_run[1] += (x[1] + x[3]) + (x[5] + x[7]);
            // ---- O^T += V^T P^T
            fp4_values<D, HPC>(ln, sta, x, na, nb, oacc);
            __syncwarp();
            if (lane == 0) mbar_arrive(ea);
            if (two) {
                fp4_values<D, HPC>(ln, stb, x + 4, na - kUnit, nb - kUnit, oacc);
                __syncwarp();
                if (lane == 0) mbar_arrive(eb);
            }
        }
        // ---- the segment's partial: lane r8 holds elements D/8 r8 .. of its two heads
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float l = l_run[j];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            const int hh = 2 * q4 + j;
            if (hh >= G) continue;
            if (split < 0 || split + span > a.max_splits) {      // cannot happen for valid lengths
                raise_error(PA_DEVERR_SEQLENS);
                continue;
            }
            const float inv = (l == 0.f ? 0.f : 1.f / l) * a.v_scale[kvh];       // a NaN stays one
            const int64_t r = ((int64_t)b * a.num_q_heads + h0 + hh) * a.max_splits + split;
            float *orow = a.o_part + r * D + r8 * (D / 8);
#pragma unroll
            for (int mt = 0; mt < KS; mt += 2)
                *reinterpret_cast<float4 *>(orow + 2 * mt) =
                    make_float4(oacc[mt][j] * inv, oacc[mt][2 + j] * inv, oacc[mt + 1][j] * inv, oacc[mt + 1][2 + j] * inv);
            if (r8 == 0) {
                a.lse_part[r] = l == 0.f ? -INFINITY : (m_run[j] + __log2f(l)) * 0.69314718055994531f;
                for (int e = 1; e < span; ++e) a.lse_part[r + e] = -INFINITY;
            }
        }
    }
}

template <int D, int HPC, bool BOX>
__global__ void __launch_bounds__((HPC + 1) * 32, Fp4Smem<D, HPC>::kCtas)
decode_fp4_kernel(const Fp4DecodeArgs a, const __grid_constant__ Fp4MapsOf<BOX> maps) {
    using S = Fp4Smem<D, HPC>;
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + S::kRing);
    uint64_t *empty = full + S::kStages;
    int32_t *prefix = reinterpret_cast<int32_t *>(empty + S::kStages);        // [B + 1]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], HPC);
        }
        fence_mbar_init();
    }
    if (!a.overlap_previous) after_previous();
    fp4_prefix(a, prefix);
    const int B = a.num_seqs;
    const int total = a.head_groups * prefix[B];
    int T = (total - 1) / (int)gridDim.x + 1;
    if (T < a.min_units) T = a.min_units;
    if (blockIdx.x == 0) {
        for (int b = threadIdx.x; b <= B; b += blockDim.x) a.ws_prefix[b] = prefix[b];
        if (threadIdx.x == 0) a.ws_header[0] = T;
    }
    const int g0 = (int)min((int64_t)blockIdx.x * T, (int64_t)total), g1 = min(total - g0, T) + g0;
    if (warp == HPC) fp4_produce<D, HPC, BOX>(a, maps, prefix, T, g0, g1, smem, full, empty, lane);
    else fp4_consume<D, HPC>(a, prefix, T, g0, g1, smem, full, empty, warp, lane);
}

// The log-sum-exp combine (decode.cu's, with its split count): W warps share a
// row's slots.  One warp per row reads 140 slots (a single long sequence) in
// 20 us, eight warps in 3; batches have rows enough and few slots each.
// A NaN among the partials stays one.
constexpr int kCombineThreads = 256;

template <int D, int W>
__global__ void __launch_bounds__(kCombineThreads) fp4_combine_kernel(
    const float *o_part, const float *lse_part, const int32_t *header, const int32_t *prefix, int32_t head_groups,
    int32_t heads_per_group, int32_t heads_per_seq, int32_t num_rows, int32_t max_splits, __nv_bfloat16 *out,
    float *lse_out) {
    constexpr int kLanes = D / 4;                    // lanes of a slot, four elements each
    constexpr int kSlots = 32 * W / kLanes;          // slots in flight
    __shared__ float top[kCombineThreads / 32], dens[kCombineThreads / kLanes];
    __shared__ float4 part[kCombineThreads];
    const int t = threadIdx.x % (32 * W), lane = t & 31;
    const int row = blockIdx.x * (kCombineThreads / (32 * W)) + threadIdx.x / (32 * W);
    after_previous();                                // the partials are complete
    int n = 0;
    if (row < num_rows) {
        const int64_t T = header[0];
        const int b = row / heads_per_seq, hg = (row % heads_per_seq) / heads_per_group;
        const int U = prefix[b + 1] - prefix[b];
        const int64_t rs = (int64_t)head_groups * prefix[b] + (int64_t)hg * U;
        n = U > 0 ? min((int)((rs + U - 1) / T - rs / T + 1), max_splits) : 0;
    }
    const float *lrow = lse_part + (int64_t)row * max_splits;
    float M = -INFINITY;
    for (int s = t; s < n; s += 32 * W) M = fmaxf(M, lrow[s]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (W > 1) {
        if (lane == 0) top[threadIdx.x >> 5] = M;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, top[(threadIdx.x >> 5) / W * W + w]);
    }
    const float *obase = o_part + (int64_t)row * max_splits * D + (t % kLanes) * 4;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float den = 0.f;
#pragma unroll 4
    for (int s = t / kLanes; s < n; s += kSlots) {
        const float l = lrow[s];
        if (l == -INFINITY) continue;                // an empty slot may hold anything
        const float w = __expf(l - M);
        const float4 x = *reinterpret_cast<const float4 *>(obase + (int64_t)s * D);
        den += w;
        acc.x += w * x.x; acc.y += w * x.y; acc.z += w * x.z; acc.w += w * x.w;
    }
    if (kSlots > 1) {                                // the lane groups' sums
        part[threadIdx.x] = acc;
        if (t % kLanes == 0) dens[threadIdx.x / kLanes] = den;
        if (W > 1) __syncthreads(); else __syncwarp();
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        den = 0.f;
        const int base = threadIdx.x - t;
#pragma unroll
        for (int g = 0; g < kSlots; ++g) {
            const float4 x = part[base + g * kLanes + t % kLanes];
            acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
            den += dens[base / kLanes + g];
        }
    }
    if (row >= num_rows || t >= kLanes) return;
    const float inv = den == 0.f ? 0.f : 1.f / den;
    *reinterpret_cast<uint2 *>(out + (int64_t)row * D + t * 4) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (lse_out != nullptr && t == 0) lse_out[row] = den == 0.f ? -INFINITY : M + __logf(den);
}

cudaError_t launch_fp4_combine(const Fp4DecodeArgs &a, const pa_decode_params &p, int heads_per_group,
                               const DecodePlan &plan, cudaStream_t stream) {
    const int rows = p.num_seqs * p.num_q_heads;
    // A CTA per row while all of them fit on the GPU at once and a row may have
    // more than a few slots.
    const bool share = plan.max_splits >= 8 && rows <= num_sms() * 8;
    const int per_block = share ? 1 : kCombineThreads / 32;
    constexpr int W = kCombineThreads / 32;
    auto kern = p.head_dim == 64 ? (share ? fp4_combine_kernel<64, W> : fp4_combine_kernel<64, 1>)
                                 : (share ? fp4_combine_kernel<128, W> : fp4_combine_kernel<128, 1>);
    const unsigned blocks = (unsigned)((rows + per_block - 1) / per_block);
    auto *out = static_cast<__nv_bfloat16 *>(p.out);
    if (a.overlap_previous) {
        // the split kernel did not wait for the kernel before it: an ordinary
        // launch waits for both
        kern<<<blocks, kCombineThreads, 0, stream>>>(a.o_part, a.lse_part, a.ws_header, a.ws_prefix, a.head_groups,
                                                     heads_per_group, p.num_q_heads, rows, plan.max_splits, out, p.lse);
        return cudaGetLastError();
    }
    return launch_after(kern, blocks, kCombineThreads, 0, stream, a.o_part, a.lse_part, a.ws_header, a.ws_prefix,
                        a.head_groups, heads_per_group, p.num_q_heads, rows, plan.max_splits, out, p.lse);
}

template <int D, int HPC, bool BOX>
cudaError_t launch_fp4_t(const Fp4DecodeArgs &a, const Fp4MapsOf<BOX> &maps, const pa_decode_params &p, int64_t useful,
                         cudaStream_t stream) {
    using S = Fp4Smem<D, HPC>;
    const size_t smem = S::kRing + 2 * S::kStages * sizeof(uint64_t) + ((size_t)a.num_seqs + 1) * sizeof(int32_t);
    auto kern = decode_fp4_kernel<D, HPC, BOX>;
    // CTAs per SM of the last (device, size), so that a serving loop's calls
    // skip both queries; the limit is raised to the device's once and for all.
    static std::atomic<uint64_t> last{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t key = ((uint64_t)(dev + 1) << 40) | ((uint64_t)smem << 8);
    int per_sm = 0;
    const uint64_t seen = last.load(std::memory_order_relaxed);
    if ((seen & ~uint64_t(255)) == key) {
        per_sm = (int)(seen & 255);
    } else {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
        if (e != cudaSuccess) return e;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, (HPC + 1) * 32, smem);
        if (e != cudaSuccess) return e;
        if (per_sm < 1) return cudaErrorInvalidConfiguration;
        last.store(key | (uint64_t)per_sm, std::memory_order_relaxed);
    }
    int64_t grid = (int64_t)num_sms() * per_sm;
    if (p.max_ctas > 0 && grid > p.max_ctas) grid = p.max_ctas;
    if (grid > useful) grid = useful;
    return launch_after(kern, (unsigned)grid, (HPC + 1) * 32, smem, stream, a, maps);
}

template <bool BOX>
cudaError_t dispatch_fp4(const Fp4DecodeArgs &a, const Fp4MapsOf<BOX> &maps, int heads, const pa_decode_params &p,
                         int64_t useful, cudaStream_t stream) {
    if (p.head_dim == 64) {
        if (heads == 1) return launch_fp4_t<64, 1, BOX>(a, maps, p, useful, stream);
        if (heads == 2) return launch_fp4_t<64, 2, BOX>(a, maps, p, useful, stream);
        if (heads == 4) return launch_fp4_t<64, 4, BOX>(a, maps, p, useful, stream);
        if (heads == 8) return launch_fp4_t<64, 8, BOX>(a, maps, p, useful, stream);
    } else {
        if (heads == 1) return launch_fp4_t<128, 1, BOX>(a, maps, p, useful, stream);
        if (heads == 2) return launch_fp4_t<128, 2, BOX>(a, maps, p, useful, stream);
        if (heads == 4) return launch_fp4_t<128, 4, BOX>(a, maps, p, useful, stream);
        if (heads == 8) return launch_fp4_t<128, 8, BOX>(a, maps, p, useful, stream);
    }
    return cudaErrorInvalidValue;
}

// 2-D map (32-bit words of a row, rows) of a 4-bit pool with a box of 16 rows
// of one head group.
bool make_map_rows(CUtensorMap *m, const void *base, const Fp4Layout &lay, int64_t rows) {
    auto enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)lay.row_bytes / 4, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)lay.row_bytes};
    cuuint32_t box[2] = {(cuuint32_t)lay.group_bytes / 4, kUnit};
    cuuint32_t es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The keys of a sequence that its query can see, up to whole units: a window
// may begin and end inside one.
int64_t reach(const pa_decode_params &p) {
    const int64_t all = ((int64_t)p.max_seqlen_k + kUnit - 1) / kUnit * kUnit;
    if (p.sliding_window <= 0) return all;
    const int64_t seen = ((int64_t)p.sliding_window + kUnit - 2) / kUnit * kUnit + kUnit;
    return seen < all ? seen : all;
}

// The automatic smallest range for `keys` a sequence: what spreads the batch at
// its longest over every SM, between 64 keys and 1/32 of the longest sequence.
int32_t smallest_range(const pa_decode_params &p, int64_t keys, int groups) {
    int64_t most = (keys / 32 + kUnit - 1) / kUnit * kUnit;
    if (most < 64) most = 64;
    const int64_t even = (p.num_seqs * keys * groups / num_sms() + kUnit - 1) / kUnit * kUnit;
    return (int32_t)(even < 64 ? 64 : even > most ? most : even);
}

// Bytes of the workspace layout (decode_setup) with `slots` partials per query head.
size_t workspace_of(const pa_decode_params &p, size_t slots) {
    const size_t rows = slots * p.num_q_heads;
    const size_t header = 256 + (((size_t)p.num_seqs + 1) * sizeof(int32_t) + 255) / 256 * 256;
    const size_t obytes = (rows * p.head_dim * sizeof(float) + 255) / 256 * 256;
    return header + obytes + rows * sizeof(float);
}

// At least the partials per query head, num_seqs * max_splits, of any batch of up
// to num_seqs sequences that see up to `keys` keys each, under smallest_range's
// ranges R.  A row has ceil(keys / R) + 1 slots, and R is 64 or more: at most
// ceil(keys / 64) + 1; and either 1/32 of the keys rounded down or more, at most 34
// slots, or at least 80 and 80/81 of num_seqs * keys * groups / SMs (a quotient
// rounded down), at most 1.0125 SMs / (groups * num_seqs) + 3.  Every bound times
// num_seqs grows with num_seqs and with keys.
size_t most_slots(const pa_decode_params &p, int64_t keys, int groups) {
    const int64_t n = p.num_seqs;
    const int64_t by_floor = n * ((keys + 63) / 64 + 1);
    const int64_t by_sms = ((int64_t)num_sms() * 81 + 80 * groups - 1) / (80 * groups) + 3 * n;
    const int64_t rest = by_sms > 34 * n ? by_sms : 34 * n;
    return (size_t)(by_floor < rest ? by_floor : rest);
}

}  // namespace

DecodePlan plan_decode_fp4(const pa_decode_params &p) {
    DecodePlan plan{};
    const Fp4Layout lay = fp4_layout(p.num_kv_heads, p.head_dim);
    plan.heads_per_cta = lay.gs;
    // With a window the ranges are those of the keys it leaves (31 sequences of
    // 14141 keys, window 15: 42 us with the ranges of 14141 keys, most CTAs idle),
    // but a row has no more of them than without it: a workspace sized without
    // the window holds both.
    const int64_t seen = reach(p);
    int64_t chunk = p.kv_chunk;
    if (chunk <= 0) {
        chunk = smallest_range(p, p.max_seqlen_k, lay.groups);
        const int64_t splits = (p.max_seqlen_k + chunk - 1) / chunk;
        if (seen < p.max_seqlen_k) {
            const int64_t fewest = ((seen + splits - 1) / splits + kUnit - 1) / kUnit * kUnit;
            chunk = smallest_range(p, seen, lay.groups);
            if (chunk < fewest) chunk = fewest;
        }
    }
    plan.kv_chunk = (int32_t)chunk;
    plan.max_splits = (int32_t)((seen + chunk - 1) / chunk) + 1;
    plan.workspace_bytes = workspace_of(p, (size_t)p.num_seqs * plan.max_splits);
    // The automatic ranges get shorter with fewer sequences and with other
    // bounds, so that a smaller batch can need more (32 query heads, 4096 keys: 4
    // sequences 2.51 MB, 3 2.63 MB); the size reported holds them all.
    plan.workspace_any = p.kv_chunk > 0 ? plan.workspace_bytes : workspace_of(p, most_slots(p, seen, lay.groups));
    return plan;
}

cudaError_t launch_decode_fp4(const pa_decode_params &p, const DecodePlan &plan, cudaStream_t stream) {
    if (p.num_seqs == 0) return cudaSuccess;
    const DecodeArgs w = decode_setup(p, plan);      // the workspace layout
    const Fp4Layout lay = fp4_layout(p.num_kv_heads, p.head_dim);
    Fp4DecodeArgs a{};
    a.q = w.q;
    a.k_cache = w.k_cache;
    a.v_cache = w.v_cache;
    a.page_table = p.page_table;
    a.pt_stride = p.page_table_stride;
    a.cache_seqlens = p.cache_seqlens;
    a.num_seqs = p.num_seqs;
    a.num_q_heads = p.num_q_heads;
    a.group = p.num_q_heads / p.num_kv_heads;
    a.page_size = p.page_size;
    a.num_pages = p.num_pages;
    a.scale_log2 = w.scale_log2;
    a.min_units = plan.kv_chunk / kUnit;
    a.max_seqlen_k = p.max_seqlen_k;
    a.max_splits = plan.max_splits;
    a.head_groups = lay.groups;
    a.row_bytes = lay.row_bytes;
    a.o_part = w.o_part;
    a.lse_part = w.lse_part;
    a.k_scale = p.k_scale;
    a.v_scale = p.v_scale;
    a.window = p.sliding_window;
    a.overlap_previous = p.overlap_previous;
    a.ws_header = w.ws_header;
    a.ws_prefix = w.ws_prefix;
    // every sequence at its longest, ranges at their smallest
    const int64_t units = reach(p) / kUnit * p.num_seqs * lay.groups;
    const int64_t useful = (units + a.min_units - 1) / a.min_units + 1;
    cudaError_t e;
    if (p.page_size == 16 && lay.groups > 1) {
        Fp4Maps maps;
        if (!make_map_rows(&maps.k, p.k_cache, lay, p.num_pages * 16) ||
            !make_map_rows(&maps.v, p.v_cache, lay, p.num_pages * 16))
            return cudaErrorNotSupported;
        e = dispatch_fp4<true>(a, maps, lay.gs, p, useful, stream);
    } else {
        e = dispatch_fp4<false>(a, Fp4NoMaps{}, lay.gs, p, useful, stream);
    }
    if (e != cudaSuccess) return e;
    return launch_fp4_combine(a, p, a.group * lay.gs, plan, stream);
}

}  // namespace pa
