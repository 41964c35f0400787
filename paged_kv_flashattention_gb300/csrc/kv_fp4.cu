// Writing and reading back a 4-bit KV pool (row layout: fp4.cuh): the
// quantising store, the rotary embedding fused with it, and the load that
// returns rows as bf16.
//
// A block is 16 consecutive elements of one head.  With g the head's scale,
//   s    = E4M3(max|x| / g / 6)          (to nearest even, at most 448)
//   code = E2M1(x / (s * g))             (to nearest even, at most 6)
// every operation an IEEE single one.  s = 0 (a block whose largest magnitude
// is below about 6 g 2^-10) stores zeros.  A NaN in a block makes its scale
// NaN, so that the whole block reads as NaN; infinities saturate.
//
// All three kernels give a lane 16 elements: two 16-byte loads, and a block's
// maximum stays inside the lane.  d/16 lanes make a head, 32 / (d/16) heads a
// unit of work; a warp takes `upw` units of one token, so that a long batch
// loads a token's cos / sin once for all its heads while a short one still
// spreads over the GPU.  The rotary gives a lane both members of its eight
// pairs; keys then change places by shuffles for the quantiser.
// Bound: long batches by the latency of their loads, which wait for the token's
// slot (and position), and by issue (8192 tokens: rotary 4.8 TB/s, store 3.6, load
// 4.4; neither issue, 56 to 64 %, nor DRAM is full), short ones by launch latency
// (2 to 4 us).
#include <cuda_bf16.h>

#include "fp4.cuh"
#include "pa_device.cuh"
#include "pa_internal.h"
#include "pdl.cuh"

namespace pa {

PA_ERROR_WORD_ACCESSOR(error_word_fp4)

namespace {

struct Fp4StoreArgs {
    const uint8_t *q;             // rotary only
    uint8_t *q_out;
    const uint8_t *k;
    const uint8_t *v;
    const int32_t *positions;
    const float *cos_sin;
    int32_t max_pos;
    int32_t rot_dim;
    int32_t interleaved;
    const int32_t *slot_mapping;
    int64_t num_tokens;
    int32_t num_q_heads;          // 0 without the rotary
    int32_t num_kv_heads;
    uint8_t *k_cache;
    uint8_t *v_cache;
    int64_t num_slots;
    const float *k_scale;
    const float *v_scale;
    Fp4Layout lay;
    int32_t upw;                  // units a warp takes
};

// Two products, two fused multiply-adds, each rounded on its own.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}" : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z, t;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 t, x, y, z;\n\tmov.b64 {%0, %1}, t;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

// Codes (8 bytes) and scale of a block of 16 bf16.
__device__ __forceinline__ void quantise16(const uint32_t (&w)[8], float g, uint2 &codes, uint32_t &scale) {
    // magnitudes of bf16 compare like the integers of their bits
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    m = max(m & 0xffffu, m >> 16);
    codes = make_uint2(0u, 0u);
    scale = 0x7f;                                    // NaN
    if (m > 0x7f80u) return;                         // a NaN in the block
    const float amax = __uint_as_float(m << 16);
    // RN(x / 6) by the division below (1/6 is rounded correctly); beyond 2688 the
    // scale is 448 anyway
    const float most = fminf(__fdiv_rn(amax, g), 65536.f);
    const float sixth = 1.f / 6.f, near6 = __fmul_rn(most, sixth);
    const float want = __fmaf_rn(__fmaf_rn(near6, 6.f, -most), -sixth, near6);
    uint16_t sc;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(sc) : "f"(0.f), "f"(want));
    scale = sc & 0xffu;
    const uint32_t s16 = e4m3x2_to_f16x2(scale);
    const float s = __low2float(*reinterpret_cast<const __half2 *>(&s16));
    const float step = __fmul_rn(s, g);
    if (!(step > 0.f)) return;
    // Sixteen divisions by one step.  With r = RN(1/step), q0 = RN(x r) and the
    // remainder e = RN(x - q0 step), q = RN(q0 + e r) rounds a number within
    // 2^-46 of the quotient (Markstein's division, IBM J. Res. Dev. 34, 1990).
    // q and RN(x/step) fall on different sides of a border t of the codes only
    // if x / step is that close to t (1 +- 2^-24); x has 8 bits and t at most
    // 3, which leaves t = 1/4 with a step whose 24 bits are all ones, and
    // there e and e r are exact.  So the codes are those of the IEEE quotient.
    // Blocks near the ends of fp32's range take the plain division.
    const float r = __frcp_rn(step);
    const bool normal = step > 1e-30f && step < 1e30f && amax < 1e30f;
    uint32_t c[2];
    const float2 r2 = make_float2(r, r), nr2 = make_float2(-r, -r), step2 = make_float2(step, step);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float2 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = make_float2(bf16lo(w[4 * h + i]), bf16hi(w[4 * h + i]));
            if (normal) {
                const float2 a = mul2(v, r2);
                // (the negative remainder times -r keeps the sign of a zero)
                x[i] = fma2(fma2(a, step2, make_float2(-v.x, -v.y)), nr2, a);
            } else {
                x[i] = make_float2(__fdiv_rn(v.x, step), __fdiv_rn(v.y, step));
            }
        }
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
            "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
            : "=r"(c[h])
            : "f"(x[0].x), "f"(x[0].y), "f"(x[1].x), "f"(x[1].y), "f"(x[2].x), "f"(x[2].y), "f"(x[3].x), "f"(x[3].y));
    }
    codes = make_uint2(c[0], c[1]);
}

// The rotary's eight pairs of a lane.  Pairs (i, i + h), h half the rotated
// width: the first rot/16 lanes of a head hold elements 8 blk .. + 7 and h + 8
// blk .. + 7.  Pairs (2i, 2i + 1): elements 16 blk .. + 15.  Lanes past the
// rotated width copy elements 16 blk .. + 15.
struct RopeLane {
    float2 c[4], s[4];            // cos and sin of pairs 2 i, 2 i + 1
    bool turn;
    int lo, hi;                   // byte offsets of the lane's two groups of eight in the head
};

__device__ __forceinline__ RopeLane rope_place(const Fp4StoreArgs &a, int blk) {
    RopeLane rl;
    rl.turn = 16 * blk < a.rot_dim;
    const bool split = rl.turn && !a.interleaved;
    rl.lo = split ? 16 * blk : 32 * blk;
    rl.hi = split ? a.rot_dim + 16 * blk : 32 * blk + 16;
    return rl;
}

__device__ __forceinline__ void rope_load(const Fp4StoreArgs &a, int pos, int blk, RopeLane &rl) {
    if (!rl.turn) return;
    const float4 *c = reinterpret_cast<const float4 *>(a.cos_sin + (int64_t)pos * a.rot_dim + 8 * blk);
    const float4 *s = reinterpret_cast<const float4 *>(a.cos_sin + (int64_t)pos * a.rot_dim + a.rot_dim / 2 + 8 * blk);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 x = c[i], y = s[i];
        rl.c[2 * i] = make_float2(x.x, x.y);
        rl.c[2 * i + 1] = make_float2(x.z, x.w);
        rl.s[2 * i] = make_float2(y.x, y.y);
        rl.s[2 * i + 1] = make_float2(y.z, y.w);
    }
}

// (a, b) -> (a c - b s, b c + a s) of the lane's pairs as the unfused rotary
// computes it: products and sum rounded in fp32, the result to bf16.
__device__ __forceinline__ void rotate16(const RopeLane &rl, bool interleaved, uint32_t (&w)[8]) {
    if (!rl.turn) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 a, b;
        if (interleaved) {
            a = make_float2(bf16lo(w[2 * i]), bf16lo(w[2 * i + 1]));
            b = make_float2(bf16hi(w[2 * i]), bf16hi(w[2 * i + 1]));
        } else {
            a = make_float2(bf16lo(w[i]), bf16hi(w[i]));
            b = make_float2(bf16lo(w[4 + i]), bf16hi(w[4 + i]));
        }
        // scalar: packed f32x2 products and sums came out fused
        const float2 c = rl.c[i], n = rl.s[i];
        const float2 x = make_float2(__fsub_rn(__fmul_rn(a.x, c.x), __fmul_rn(b.x, n.x)),
                                     __fsub_rn(__fmul_rn(a.y, c.y), __fmul_rn(b.y, n.y)));
        const float2 y = make_float2(__fadd_rn(__fmul_rn(b.x, c.x), __fmul_rn(a.x, n.x)),
                                     __fadd_rn(__fmul_rn(b.y, c.y), __fmul_rn(a.y, n.y)));
        if (interleaved) {
            w[2 * i] = pack_bf16x2(x.x, y.x);
            w[2 * i + 1] = pack_bf16x2(x.y, y.y);
        } else {
            w[i] = pack_bf16x2(x.x, x.y);
            w[4 + i] = pack_bf16x2(y.x, y.y);
        }
    }
}

// From the places of pairs (i, i + h) to 16 consecutive elements per lane (the
// quantiser's blocks).  Every lane of the warp calls it; `first` is the head's
// first lane.
__device__ __forceinline__ void regroup16(const Fp4StoreArgs &a, int first, int blk, uint32_t (&w)[8]) {
    const int half = a.rot_dim / 16;                 // groups of eight of the first elements; lanes that turn
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int g = 2 * blk + j;                   // the group wanted
        const int src = first + (g < half ? g : g < 2 * half ? g - half : g >> 1);
        const bool second = g < half ? false : g < 2 * half ? true : g & 1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = __shfl_sync(0xffffffffu, w[i], src), y = __shfl_sync(0xffffffffu, w[4 + i], src);
            o[4 * j + i] = second ? y : x;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = o[i];
}

// UG: units whose loads go out together.  The rotary on 8192 tokens (32 + 8
// heads of 128, 178 MB): two units at 64 registers 38.0 us; earlier, when that
// was 38.8, at 80 44.0, at 106 53.5, one unit at 64 41.8, four at 123 50.9.  When a lane held 16 consecutive
// elements and fetched their partners through memory it was 63 us, by shuffles
// 49.  The plain store of the same tokens (43 MB) is 12.1 us with one unit, 12.4
// with two; 14.0 before its products were packed by two.
template <int D, bool ROPE, int UG>
__global__ void __launch_bounds__(256, 4) fp4_store_kernel(const Fp4StoreArgs a) {
    constexpr int kLanes = D / 16;                   // lanes of a head
    constexpr int kHeads = 32 / kLanes;              // heads of a unit
    after_previous();
    const int lane = threadIdx.x & 31;
    const int blk = lane % kLanes, sub = lane / kLanes;
    const int uq = (a.num_q_heads + kHeads - 1) / kHeads, uk = (a.num_kv_heads + kHeads - 1) / kHeads;
    const int units = uq + 2 * uk;
    const int parts = (units + a.upw - 1) / a.upw;   // warps of a token
    const bool inter = a.interleaved != 0;
    const int64_t warps_total = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t i = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); i < a.num_tokens * parts;
         i += warps_total) {
        const int64_t t = i / parts;
        const int u0 = (int)(i - t * parts) * a.upw, u1 = min(u0 + a.upw, units);
        const int slot = a.slot_mapping[t];
        const bool store = slot >= 0 && slot < a.num_slots;
        if (u0 == 0 && slot >= a.num_slots && lane == 0) raise_error(PA_DEVERR_PAGE_RANGE);
        RopeLane rl;
        if (ROPE) {
            const int pos = a.positions[t];
            if (pos < 0 || pos >= a.max_pos) {       // nothing of this token is written
                if (u0 == 0 && lane == 0) raise_error(PA_DEVERR_POSITION);
                continue;
            }
            rl = rope_place(a, blk);
            rope_load(a, pos, blk, rl);
        } else if (!store) {
            continue;
        }
        for (int u = u0; u < u1; u += UG) {
            uint32_t w[UG][8];
            int off[UG];                             // the head's byte offset in its token; -1: no such head
#pragma unroll
            for (int g = 0; g < UG; ++g) {           // q, then k, then v
                const int n = u + g;
                const bool is_q = n < uq, is_k = n < uq + uk;
                const int h = (is_q ? n : n - uq - (is_k ? 0 : uk)) * kHeads + sub;
                const int heads = is_q ? a.num_q_heads : a.num_kv_heads;
                off[g] = n < u1 && h < heads && (is_q || store) ? h * (2 * D) : -1;
#pragma unroll
                for (int e = 0; e < 8; ++e) w[g][e] = 0u;
                if (off[g] < 0) continue;
                const uint8_t *head = (is_q ? a.q : is_k ? a.k : a.v) + t * heads * (2 * D) + off[g];
                const bool pairs = ROPE && is_k;
                const uint4 x = *reinterpret_cast<const uint4 *>(head + (pairs ? rl.lo : 32 * blk));
                const uint4 y = *reinterpret_cast<const uint4 *>(head + (pairs ? rl.hi : 32 * blk + 16));
                w[g][0] = x.x; w[g][1] = x.y; w[g][2] = x.z; w[g][3] = x.w;
                w[g][4] = y.x; w[g][5] = y.y; w[g][6] = y.z; w[g][7] = y.w;
            }
#pragma unroll
            for (int g = 0; g < UG; ++g) {
                const int n = u + g;
                if (n >= u1) break;
                const bool is_q = n < uq, is_k = n < uq + uk;
                if (ROPE && is_k) rotate16(rl, inter, w[g]);
                if (is_q) {                          // (in place too: a lane writes what it alone read)
                    if (off[g] < 0) continue;
                    uint8_t *dst = a.q_out + t * a.num_q_heads * (2 * D) + off[g];
                    *reinterpret_cast<uint4 *>(dst + rl.lo) = make_uint4(w[g][0], w[g][1], w[g][2], w[g][3]);
                    *reinterpret_cast<uint4 *>(dst + rl.hi) = make_uint4(w[g][4], w[g][5], w[g][6], w[g][7]);
                    continue;
                }
                if (ROPE && is_k && !inter) regroup16(a, lane - blk, blk, w[g]);
                if (off[g] < 0) continue;
                const int h = off[g] / (2 * D);
                uint2 codes;
                uint32_t scale;
                quantise16(w[g], (is_k ? a.k_scale : a.v_scale)[h], codes, scale);
                const int hg = h & (a.lay.gs - 1);   // gs is a power of two
                uint8_t *row = (is_k ? a.k_cache : a.v_cache) + (int64_t)slot * a.lay.row_bytes +
                               (h / a.lay.gs) * a.lay.group_bytes;
                *reinterpret_cast<uint2 *>(row + hg * (D / 2) + blk * 8) = codes;
                row[a.lay.code_bytes + hg * kLanes + blk] = (uint8_t)scale;
            }
        }
    }
}

// Rows back as bf16: code * block scale is exact, times the head's scale
// rounded in fp32, then to bf16.  8192 rows of 8 heads of 128 (43 MB): 9.7 us;
// with half the units per warp 8.7, but 5.9 instead of 4.9 on rows of 3 heads of
// 64.
template <int D>
__global__ void __launch_bounds__(256) fp4_load_kernel(const int32_t *slots, int64_t num_tokens,
                                                       const uint8_t *k_cache, const uint8_t *v_cache,
                                                       int64_t num_slots, int32_t num_kv_heads,
                                                       const float *k_scale, const float *v_scale, uint8_t *k_out,
                                                       uint8_t *v_out, Fp4Layout lay, int32_t upw) {
    constexpr int kLanes = D / 16, kHeads = 32 / kLanes;
    after_previous();
    const int lane = threadIdx.x & 31;
    const int blk = lane % kLanes, sub = lane / kLanes;
    const int uk = (num_kv_heads + kHeads - 1) / kHeads, units = 2 * uk;
    const int parts = (units + upw - 1) / upw;
    const int64_t warps_total = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t i = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); i < num_tokens * parts;
         i += warps_total) {
        const int64_t t = i / parts;
        const int u0 = (int)(i - t * parts) * upw, u1 = min(u0 + upw, units);
        const int64_t slot = slots[t];
        const bool live = slot >= 0 && slot < num_slots;
        if (slot >= num_slots && lane == 0) raise_error(PA_DEVERR_PAGE_RANGE);
        for (int u = u0; u < u1; ++u) {
            const bool is_k = u < uk;
            const int h = (u - (is_k ? 0 : uk)) * kHeads + sub;
            if (h >= num_kv_heads) continue;
            uint32_t o[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
            if (live) {
                const int hg = h & (lay.gs - 1);
                const uint8_t *row = (is_k ? k_cache : v_cache) + slot * lay.row_bytes + (h / lay.gs) * lay.group_bytes;
                const uint2 codes = *reinterpret_cast<const uint2 *>(row + hg * (D / 2) + blk * 8);
                const uint32_t s = f16_dup_lo(e4m3x2_to_f16x2(row[lay.code_bytes + hg * kLanes + blk]));
                const float g = (is_k ? k_scale : v_scale)[h];
                uint32_t r[8];
                e2m1x8_to_f16x8(codes.x, *reinterpret_cast<uint32_t(*)[4]>(&r[0]));
                e2m1x8_to_f16x8(codes.y, *reinterpret_cast<uint32_t(*)[4]>(&r[4]));
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t x = hmul2_bits(r[j], s);
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x));
                    o[j] = pack_bf16x2(f.x * g, f.y * g);
                }
            }
            uint4 *dst = reinterpret_cast<uint4 *>((is_k ? k_out : v_out) + ((t * num_kv_heads + h) * D + blk * 16) * 2);
            dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
            dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
}

// Units a warp takes, and the grid: at least 32 warps' worth of work per SM
// before a warp takes a second unit, never more than a whole token.
struct StoreGrid {
    int32_t upw;
    unsigned blocks;
};
StoreGrid store_grid(int64_t tokens, int units) {
    const int64_t want = (int64_t)num_sms() * 32;
    int64_t parts = (want + tokens - 1) / tokens;    // warps of a token
    if (parts > units) parts = units;
    const int upw = (int)((units + parts - 1) / parts);
    const int64_t warps = tokens * ((units + upw - 1) / upw);
    int64_t blocks = (warps + 7) / 8;
    const int64_t cap = (int64_t)num_sms() * 16;
    if (blocks > cap) blocks = cap;
    return {upw, (unsigned)blocks};
}

template <bool ROPE>
cudaError_t launch_store_t(Fp4StoreArgs &a, int d, cudaStream_t stream) {
    const int heads = 32 / (d / 16);
    const int units = (a.num_q_heads + heads - 1) / heads + 2 * ((a.num_kv_heads + heads - 1) / heads);
    const StoreGrid g = store_grid(a.num_tokens, units);
    a.upw = g.upw;
    constexpr int UG = ROPE ? 2 : 1;
    auto kern = d == 64 ? fp4_store_kernel<64, ROPE, UG> : fp4_store_kernel<128, ROPE, UG>;
    return launch_after(kern, g.blocks, 256, 0, stream, a);
}

}  // namespace

cudaError_t launch_store_kv_fp4(const void *k, const void *v, const int32_t *slot_mapping, int64_t num_tokens,
                                void *k_cache, void *v_cache, int64_t num_slots, int32_t num_kv_heads,
                                int32_t head_dim, const float *k_scale, const float *v_scale, cudaStream_t stream) {
    Fp4StoreArgs a{};
    a.k = static_cast<const uint8_t *>(k);
    a.v = static_cast<const uint8_t *>(v);
    a.slot_mapping = slot_mapping;
    a.num_tokens = num_tokens;
    a.num_kv_heads = num_kv_heads;
    a.k_cache = static_cast<uint8_t *>(k_cache);
    a.v_cache = static_cast<uint8_t *>(v_cache);
    a.num_slots = num_slots;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.lay = fp4_layout(num_kv_heads, head_dim);
    return launch_store_t<false>(a, head_dim, stream);
}

cudaError_t launch_rope_store_fp4(const pa_rope_store_params &p, cudaStream_t stream) {
    Fp4StoreArgs a{};
    a.q = static_cast<const uint8_t *>(p.q);
    a.q_out = static_cast<uint8_t *>(p.q_out);
    a.k = static_cast<const uint8_t *>(p.k);
    a.v = static_cast<const uint8_t *>(p.v);
    a.positions = p.positions;
    a.cos_sin = p.cos_sin;
    a.max_pos = p.max_pos;
    a.rot_dim = p.rot_dim;
    a.interleaved = p.interleaved;
    a.slot_mapping = p.slot_mapping;
    a.num_tokens = p.num_tokens;
    a.num_q_heads = p.num_q_heads;
    a.num_kv_heads = p.num_kv_heads;
    a.k_cache = static_cast<uint8_t *>(p.k_cache);
    a.v_cache = static_cast<uint8_t *>(p.v_cache);
    a.num_slots = p.num_slots;
    a.k_scale = p.k_scale;
    a.v_scale = p.v_scale;
    a.lay = fp4_layout(p.num_kv_heads, p.head_dim);
    return launch_store_t<true>(a, p.head_dim, stream);
}

cudaError_t launch_load_kv_fp4(const int32_t *slots, int64_t num_tokens, const void *k_cache, const void *v_cache,
                               int64_t num_slots, int32_t num_kv_heads, int32_t head_dim, const float *k_scale,
                               const float *v_scale, void *k_out, void *v_out, cudaStream_t stream) {
    const int heads = 32 / (head_dim / 16);
    const StoreGrid g = store_grid(num_tokens, 2 * ((num_kv_heads + heads - 1) / heads));
    auto kern = head_dim == 64 ? fp4_load_kernel<64> : fp4_load_kernel<128>;
    return launch_after(kern, g.blocks, 256, 0, stream, slots, num_tokens, static_cast<const uint8_t *>(k_cache),
                        static_cast<const uint8_t *>(v_cache), num_slots, num_kv_heads, k_scale, v_scale,
                        static_cast<uint8_t *>(k_out), static_cast<uint8_t *>(v_out), fp4_layout(num_kv_heads, head_dim),
                        g.upw);
}

}  // namespace pa
