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
// All three kernels give a lane one block: 16 elements are two 16-byte loads,
// and the block's maximum stays inside the lane.  d/16 lanes make a head,
// 32 / (d/16) heads a unit of work; a warp takes `upw` units of one token, so
// that a long batch loads a token's cos / sin once for all its heads while a
// short one still spreads over the GPU.
// Bound: HBM for long batches (per element 2 bytes in, 9/16 out), launch
// latency for short ones.
#include <cuda_bf16.h>

#include "fp4.cuh"
#include "pa_device.cuh"
#include "pa_internal.h"

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

__device__ __forceinline__ void load16(const uint8_t *p, uint32_t (&w)[8]) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p), b = *reinterpret_cast<const uint4 *>(p + 16);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
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
    const float want = __fdiv_rn(__fdiv_rn(amax, g), 6.f);
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
    uint32_t c[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float lo = bf16lo(w[i]), hi = bf16hi(w[i]);
        float a, b;
        if (normal) {
            a = __fmul_rn(lo, r);
            b = __fmul_rn(hi, r);
            // (written with -e, which keeps the sign of a zero)
            a = __fmaf_rn(-__fmaf_rn(a, step, -lo), r, a);
            b = __fmaf_rn(-__fmaf_rn(b, step, -hi), r, b);
        } else {
            a = __fdiv_rn(lo, step);
            b = __fdiv_rn(hi, step);
        }
        uint32_t two;
        asm("{\n\t.reg .b8 t;\n\t.reg .b16 x;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\t"
            "mov.b16 x, {t, t};\n\tcvt.u32.u16 %0, x;\n\t}" : "=r"(two) : "f"(b), "f"(a));
        c[i >> 2] |= (two & 0xffu) << (8 * (i & 3));
    }
    codes = make_uint2(c[0], c[1]);
}

// The lane's cos and sin: group j (elements 8 w .. 8 w + 7 of a head, w = 2 blk
// + j) becomes own * c + partner * s, the sign of the rotation inside s.
struct RopeLane {
    float c[2][8], s[2][8];
    int partner[2];               // byte offset of the partner group within the head; -1: not rotated
};

__device__ __forceinline__ void rope_lane(const Fp4StoreArgs &a, int pos, int blk, RopeLane &rl) {
    const int rot = a.rot_dim, h = rot / 2;
    const float *row = a.cos_sin + (int64_t)pos * rot;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int e = 16 * blk + 8 * j;
        rl.partner[j] = -1;
        if (e >= rot) continue;
        if (a.interleaved) {
            rl.partner[j] = 2 * e;                       // pairs lie inside the group
            const float4 c = *reinterpret_cast<const float4 *>(row + e / 2);
            const float4 s = *reinterpret_cast<const float4 *>(row + h + e / 2);
            const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                rl.c[j][2 * i] = rl.c[j][2 * i + 1] = cv[i];
                rl.s[j][2 * i] = -sv[i];
                rl.s[j][2 * i + 1] = sv[i];
            }
        } else {
            const bool first = e < h;
            const int i0 = first ? e : e - h;
            rl.partner[j] = 2 * (first ? e + h : e - h);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 c = *reinterpret_cast<const float4 *>(row + i0 + 4 * i);
                const float4 s = *reinterpret_cast<const float4 *>(row + h + i0 + 4 * i);
                rl.c[j][4 * i] = c.x; rl.c[j][4 * i + 1] = c.y; rl.c[j][4 * i + 2] = c.z; rl.c[j][4 * i + 3] = c.w;
                const float f = first ? -1.f : 1.f;
                rl.s[j][4 * i] = f * s.x; rl.s[j][4 * i + 1] = f * s.y;
                rl.s[j][4 * i + 2] = f * s.z; rl.s[j][4 * i + 3] = f * s.w;
            }
        }
    }
}

// Rotate the lane's block w of the head at `head` (16 bf16), as the unfused
// rotary does: products and sum rounded in fp32, the result to bf16.
__device__ __forceinline__ void rotate16(const Fp4StoreArgs &a, const RopeLane &rl, const uint8_t *head, uint32_t (&w)[8]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (rl.partner[j] < 0) continue;
        uint32_t p[4];
        if (a.interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = __byte_perm(w[4 * j + i], 0u, 0x1032);
        } else {
            const uint4 x = *reinterpret_cast<const uint4 *>(head + rl.partner[j]);
            p[0] = x.x; p[1] = x.y; p[2] = x.z; p[3] = x.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t o = w[4 * j + i];
            const float lo = __fadd_rn(__fmul_rn(bf16lo(o), rl.c[j][2 * i]), __fmul_rn(bf16lo(p[i]), rl.s[j][2 * i]));
            const float hi = __fadd_rn(__fmul_rn(bf16hi(o), rl.c[j][2 * i + 1]), __fmul_rn(bf16hi(p[i]), rl.s[j][2 * i + 1]));
            p[i] = pack_bf16x2(lo, hi);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) w[4 * j + i] = p[i];
    }
}

template <int D, bool ROPE>
__global__ void __launch_bounds__(256) fp4_store_kernel(const Fp4StoreArgs a) {
    constexpr int kLanes = D / 16;                   // lanes of a head
    constexpr int kHeads = 32 / kLanes;              // heads of a unit
    const int lane = threadIdx.x & 31;
    const int blk = lane % kLanes, sub = lane / kLanes;
    const int uq = (a.num_q_heads + kHeads - 1) / kHeads, uk = (a.num_kv_heads + kHeads - 1) / kHeads;
    const int units = uq + 2 * uk;
    const int parts = (units + a.upw - 1) / a.upw;   // warps of a token
    const int64_t warps_total = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t i = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); i < a.num_tokens * parts;
         i += warps_total) {
        const int64_t t = i / parts;
        const int u0 = (int)(i - t * parts) * a.upw, u1 = min(u0 + a.upw, units);
        const int64_t slot = a.slot_mapping[t];
        const bool store = slot >= 0 && slot < a.num_slots;
        if (slot >= a.num_slots && lane == 0) raise_error(PA_DEVERR_PAGE_RANGE);
        RopeLane rl;
        if (ROPE) {
            const int pos = a.positions[t];
            if (pos < 0 || pos >= a.max_pos) {       // nothing of this token is written
                if (lane == 0) raise_error(PA_DEVERR_POSITION);
                continue;
            }
            rope_lane(a, pos, blk, rl);
        } else if (!store) {
            continue;
        }
        for (int u = u0; u < u1; ++u) {
            if (ROPE && u < uq) {
                const int h = u * kHeads + sub;
                const int64_t off = ((t * a.num_q_heads + h) * D) * 2;
                uint32_t w[8];
                if (h < a.num_q_heads) {
                    load16(a.q + off + blk * 32, w);
                    rotate16(a, rl, a.q + off, w);
                }
                __syncwarp();                        // q_out may be q: every partner is read first
                if (h < a.num_q_heads) {
                    uint4 *dst = reinterpret_cast<uint4 *>(a.q_out + off + blk * 32);
                    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
                    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
                }
                continue;
            }
            const bool is_k = u < uq + uk;
            const int h = (u - uq - (is_k ? 0 : uk)) * kHeads + sub;
            if (!store || h >= a.num_kv_heads) continue;
            const uint8_t *head = (is_k ? a.k : a.v) + ((t * a.num_kv_heads + h) * D) * 2;
            uint32_t w[8];
            load16(head + blk * 32, w);
            if (ROPE && is_k) rotate16(a, rl, head, w);
            uint2 codes;
            uint32_t scale;
            quantise16(w, __ldg((is_k ? a.k_scale : a.v_scale) + h), codes, scale);
            const int hg = h & (a.lay.gs - 1);       // gs is a power of two
            uint8_t *row = (is_k ? a.k_cache : a.v_cache) + slot * a.lay.row_bytes + (h / a.lay.gs) * a.lay.group_bytes;
            *reinterpret_cast<uint2 *>(row + hg * (D / 2) + blk * 8) = codes;
            row[a.lay.code_bytes + hg * kLanes + blk] = (uint8_t)scale;
        }
    }
}

// Rows back as bf16: code * block scale is exact, times the head's scale
// rounded in fp32, then to bf16.
template <int D>
__global__ void __launch_bounds__(256) fp4_load_kernel(const int32_t *__restrict__ slots, int64_t num_tokens,
                                                       const uint8_t *__restrict__ k_cache,
                                                       const uint8_t *__restrict__ v_cache, int64_t num_slots,
                                                       int32_t num_kv_heads, const float *__restrict__ k_scale,
                                                       const float *__restrict__ v_scale, uint8_t *k_out,
                                                       uint8_t *v_out, Fp4Layout lay, int32_t upw) {
    constexpr int kLanes = D / 16, kHeads = 32 / kLanes;
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
                const float g = __ldg((is_k ? k_scale : v_scale) + h);
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
    int64_t upw = tokens * units / want;
    if (upw < 1) upw = 1;
    if (upw > units) upw = units;
    const int64_t warps = tokens * ((units + upw - 1) / upw);
    int64_t blocks = (warps + 7) / 8;
    const int64_t cap = (int64_t)num_sms() * 16;
    if (blocks > cap) blocks = cap;
    return {(int32_t)upw, (unsigned)blocks};
}

template <bool ROPE>
cudaError_t launch_store_t(Fp4StoreArgs &a, int d, cudaStream_t stream) {
    const int heads = 32 / (d / 16);
    const int units = (a.num_q_heads + heads - 1) / heads + 2 * ((a.num_kv_heads + heads - 1) / heads);
    const StoreGrid g = store_grid(a.num_tokens, units);
    a.upw = g.upw;
    if (d == 64) fp4_store_kernel<64, ROPE><<<g.blocks, 256, 0, stream>>>(a);
    else fp4_store_kernel<128, ROPE><<<g.blocks, 256, 0, stream>>>(a);
    return cudaGetLastError();
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
    kern<<<g.blocks, 256, 0, stream>>>(slots, num_tokens, static_cast<const uint8_t *>(k_cache),
                                       static_cast<const uint8_t *>(v_cache), num_slots, num_kv_heads, k_scale, v_scale,
                                       static_cast<uint8_t *>(k_out), static_cast<uint8_t *>(v_out),
                                       fp4_layout(num_kv_heads, head_dim), g.upw);
    return cudaGetLastError();
}

}  // namespace pa
