// Decode over shared prefixes: sequences in groups (the beams or samples of one
// request, requests behind one system prompt) whose first keys are the same.
//
//   out[b, h] = softmax over keys [0, L_b) of (scale q[b, h] . K) V
//
// splits at the prefix P of b's group (log-sum-exp, "Transformer inference
// kernels (3/10)", sections 12 and 16): keys [0, P) are read once for the whole
// group, keys [P, L_b) by the split-KV decode, and one merge joins a row's
// partials of both.
//
// The prefix is a matrix product again: the rows that read KV head kvh of a
// group are (sequence, query head of kvh), n * Hq / Hkv of them, so prefill's
// tcgen05 kernel does it (prefill_impl.cuh, SHARED) with tiles of 128 such rows,
// two tiles per CTA (over FP8 and 4-bit pools one); where a group fills only one,
// the tile's key steps go in turn to two softmax halves, each with partials of its
// own.  Query rows come in tensor-map boxes of 32 (64 columns, Hq / Hkv heads,
// 32 Hkv / Hq sequences).
// Every CTA gets the same number of 128-key steps, whatever the groups are; the
// partials are written in 32 bits, a block of 8 warps' 32 rows for each work item.
// The decode of the other keys runs beside it, on the SMs it leaves (shared_ctas).
#include "prefill_impl.cuh"

#include <atomic>

#include "pdl.cuh"

namespace pa {

PA_ERROR_WORD_ACCESSOR(error_word_decode_shared)

namespace {

constexpr int prefix_threads(int kv) { return shared_threads(kv != PA_KV_BF16, kv == PA_KV_FP4); }

template <int D, int KV>
__global__ void __launch_bounds__(prefix_threads(KV), 1) shared_prefix_kernel(const __grid_constant__ PrefillArgs a) {
    prefill_body<D, 2, KV != PA_KV_BF16, false, KV == PA_KV_FP4, true>(a);
}

template <int D, int KV>
cudaError_t launch_prefix_t(const PrefillArgs &a, unsigned ctas, cudaStream_t stream) {
    using S = PrefillSmem<D, 2, KV != PA_KV_BF16, KV == PA_KV_FP4, true>;
    // three slots for the MMAs: K of the next step of a tile's other half beside
    // K and V of this one
    static_assert(S::kSlots >= 3 && (KV == PA_KV_BF16 || S::kCSlots >= 3), "ring too small");
    static_assert(S::kTotal + 1024 <= 232448, "shared memory");
    // One CTA per SM (it allocates all 512 TMEM columns).
    const int smem = (S::kTotal + 1024) > 120 * 1024 ? (S::kTotal + 1024) : 120 * 1024;
    auto kern = shared_prefix_kernel<D, KV>;
    static std::atomic<uint64_t> ready{0};           // devices on which the kernel may use that much, of the first 64
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if ((ready.load(std::memory_order_relaxed) & bit) == 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    return launch_after(kern, ctas, prefix_threads(KV), smem, stream, a);
}

template <int KV>
cudaError_t launch_prefix(const PrefillArgs &a, int d, unsigned ctas, cudaStream_t stream) {
    return d == 128 ? launch_prefix_t<128, KV>(a, ctas, stream) : launch_prefix_t<64, KV>(a, ctas, stream);
}

constexpr int kBlockRows = 2 * kBM;                  // rows of a block of partials: 8 softmax warps' 32
// Query rows of a work item of the prefix kernel (PrefillSmem::kItemTiles tiles).
constexpr int item_rows(int kv_dtype) { return kv_dtype == PA_KV_BF16 ? 2 * kBM : kBM; }

struct MergeArgs {
    SharedArgs sh;
    DecodeTail tail;              // o_part null: no keys behind the prefixes
    const int32_t *cache_seqlens;
    int32_t num_seqs;
    int32_t num_q_heads;
    int32_t num_kv_heads;
    int32_t max_seqlen_k;
    int32_t item_rows;
    __nv_bfloat16 *out;
    float *lse;
};

// The group of sequence b (the last g with cu_groups[g] <= b), by a whole warp:
// 32 probes a step.  num_groups for sequences behind the last group, -1 before
// the first.
__device__ __forceinline__ int group_of(const SharedArgs &sh, int b, int lane) {
    int lo = 0, n = sh.num_groups + 1;
    for (;;) {
        const int step = (n + 31) / 32;
        const int i = lane * step;
        const unsigned m = __ballot_sync(0xffffffffu, i < n && sh.cu_groups[lo + i] <= b);
        if (m == 0) return lo - 1;                   // (only in the first step)
        const int last = 31 - __clz(m);
        lo += last * step;
        n = min(step, n - last * step);
        if (step == 1) return lo;
    }
}

// One row (sequence, query head) of both lists of partials, merged by
// log-sum-exp.  W warps share a row; warp w takes slots w, w + W, .., 32 at a
// time: a lane reads one slot's lse and holds its weight, then the warp reads the
// slots that have any, kBatch of them in flight.  A NaN among the partials stays one.
constexpr int kMergeThreads = 256;
constexpr int kBatch = 8;

template <int D, int W>
__global__ void __launch_bounds__(kMergeThreads) shared_merge_kernel(const MergeArgs a) {
    constexpr int E = D / 32;                        // elements of a lane
    __shared__ float tops[kMergeThreads / 32], dens[kMergeThreads / 32];
    __shared__ float parts[W > 1 ? kMergeThreads / 32 : 1][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = warp % W;
    const int64_t num_rows = (int64_t)a.num_seqs * a.num_q_heads;
    const int64_t given = (int64_t)blockIdx.x * (kMergeThreads / (32 * W)) + warp / W;
    const int64_t row = given < num_rows ? given : num_rows - 1;
    const int b = (int)(row / a.num_q_heads), h = (int)(row % a.num_q_heads);
    const int group = a.num_q_heads / a.num_kv_heads;
    after_previous();                                // the partials are complete
    // what does not depend on one another is read together
    const int L = a.cache_seqlens[b], P = a.sh.prefix_lens[b];
    const bool has_tail = a.tail.o_part != nullptr;
    const int T = has_tail ? a.tail.header[0] : 1, u0 = has_tail ? a.tail.prefix[b] : 0, u1 = has_tail ? a.tail.prefix[b + 1] : 0;
    const int per = a.sh.header != nullptr ? a.sh.header[0] : 1;
    const int g = a.sh.header != nullptr ? group_of(a.sh, b, lane) : -1;
    bool ok = L >= 0 && L <= a.max_seqlen_k && P >= 0 && P <= L && P <= a.sh.max_prefix;
    int np = 0, ns = 0;                              // partials of the prefix, of the keys behind it
    // Partial s of the prefix: range s / each, half s % each (of a single tile), at row
    // `first` of lse_part and o_part for s = 0.
    int each = 1, apart = 0;                         // partials of a range, rows between them
    int64_t first = 0;
    if (ok && P > 0) {
        ok = g >= 0 && g < a.sh.num_groups;          // else a prefix without a group
        if (ok) {
            const int q0 = a.sh.cu_groups[g], n = a.sh.cu_groups[g + 1] - q0;
            const int2 base = a.sh.base[g];
            ok = q0 >= 0 && n <= a.sh.max_group && a.sh.prefix_lens[q0] == P;
            const int tiles = (n * group + a.item_rows - 1) / a.item_rows, steps = (P + kBN - 1) / kBN;
            const int in_group = (b - q0) * group + h % group, tile = in_group / a.item_rows, m = in_group % a.item_rows;
            const int row = (h / group) * tiles + tile, start = base.x + row * (steps + kItemSteps) + kItemSteps;
            const int rows = min(n * group - tile * a.item_rows, a.item_rows);
            const int c0 = start / per, block = c0 + base.y + row;
            const int ranges = min((start + steps - 1) / per - c0 + 1, a.sh.max_blocks - block);
            if (rows <= kBM) {                       // two halves, the second in the upper lanes where they are free
                each = 2;
                apart = rows <= kBM / 2 ? kBM + kBM / 2 : kBM;
            }
            if (ok) np = max(ranges, 0) * each;
            first = (int64_t)block * kBlockRows + m;
        }
    } else if (ok && L > 0 && g >= 0 && g < a.sh.num_groups) {
        const int q0 = a.sh.cu_groups[g];            // none, in a group that has one (the result is right all the same)
        if (q0 >= 0 && a.sh.prefix_lens[q0] != 0 && lane == 0) raise_error(PA_DEVERR_SEQLENS);
    }
    if (ok && has_tail) {
        const int U = u1 - u0;
        const int rs = a.tail.head_groups * u0 + (h / a.tail.heads_per_group) * U;
        ns = U > 0 ? min((int)(((int64_t)rs + U - 1) / T) - rs / T + 1, a.tail.max_splits) : 0;
    } else if (L > P) {
        ok = false;                                  // the call allows no keys behind the prefix
    }
    if (!ok && L != 0 && lane == 0) raise_error(PA_DEVERR_SEQLENS);
    const int n = ok ? np + ns : 0;
    const int shift = __ffs(each) - 1;
    auto at_of = [&](int s) { return first + (int64_t)(s >> shift) * kBlockRows + (s & (each - 1)) * apart; };
    const float *ls = a.tail.lse_part + row * a.tail.max_splits - np;
    const float *os = a.tail.o_part + (row * a.tail.max_splits - np) * D + lane * E;
    auto lse_of = [&](int s) { return s >= n ? -INFINITY : s < np ? a.sh.lse_part[at_of(s)] : ls[s]; };
    const int mine = w + lane * W;                   // this lane's slot of the first 32
    const float l0 = lse_of(mine);
    float M = l0;
    for (int s = mine + 32 * W; s < n; s += 32 * W) M = fmaxf(M, lse_of(s));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (W > 1) {
        if (lane == 0) tops[warp] = M;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < W; ++i) M = fmaxf(M, tops[warp - w + i]);
    }
    float acc[E], den = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int s0 = 0; s0 < n; s0 += 32 * W) {
        const float l = s0 == 0 ? l0 : lse_of(s0 + mine);
        const float wt = l == -INFINITY ? 0.f : __expf(l - M);       // an empty slot may hold anything
        den += wt;
        unsigned live = __ballot_sync(0xffffffffu, wt != 0.f);
        while (live != 0u) {
            float v[kBatch][E], f[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int at = live != 0u ? __ffs(live) - 1 : 32;
                live &= live - 1u;
                f[i] = __shfl_sync(0xffffffffu, wt, at & 31);
                if (at == 32) f[i] = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) v[i][e] = 0.f;
                if (at == 32) continue;              // the same on every lane
                const int s = s0 + w + at * W;
                const float *from = s < np ? a.sh.o_part + at_of(s) * D + lane * E : os + (int64_t)s * D;
                if constexpr (E == 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(from);
                    v[i][0] = x.x; v[i][1] = x.y; v[i][2] = x.z; v[i][3] = x.w;
                } else {
                    const float2 x = *reinterpret_cast<const float2 *>(from);
                    v[i][0] = x.x; v[i][1] = x.y;
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] += f[i] * v[i][e];
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    if (W > 1) {
        if (lane == 0) dens[warp] = den;
#pragma unroll
        for (int e = 0; e < E; ++e) parts[W > 1 ? warp : 0][lane * E + e] = acc[e];
        __syncthreads();
        if (w != 0) return;
        den = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            den += dens[warp + i];
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += parts[W > 1 ? warp + i : 0][lane * E + e];
        }
    }
    if (given >= num_rows) return;
    const float inv = den == 0.f ? 0.f : 1.f / den;
    __nv_bfloat16 *to = a.out + row * D + lane * E;
    if constexpr (E == 4)
        *reinterpret_cast<uint2 *>(to) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
    else
        *reinterpret_cast<uint32_t *>(to) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    if (a.lse != nullptr && lane == 0) a.lse[row] = den == 0.f ? -INFINITY : M + __logf(den);
}

cudaError_t launch_merge(const MergeArgs &a, int d, cudaStream_t stream) {
    const int64_t rows = (int64_t)a.num_seqs * a.num_q_heads;
    // A CTA per row while all of them fit on the GPU at once: rows of few sequences
    // have the most partials.
    constexpr int W = kMergeThreads / 32;
    const bool share = rows <= num_sms() * 8;
    const int per_block = share ? 1 : W;
    auto kern = d == 64 ? (share ? shared_merge_kernel<64, W> : shared_merge_kernel<64, 1>)
                        : (share ? shared_merge_kernel<128, W> : shared_merge_kernel<128, 1>);
    return launch_after(kern, (unsigned)((rows + per_block - 1) / per_block), kMergeThreads, 0, stream, a);
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// 3-D bf16 map of q (d, Hq, sequences) with a box of 32 rows: `group` heads of
// 32 / group sequences.
bool make_map_shared_q(CUtensorMap *m, const pa_decode_params &p) {
    auto enc = encoder();
    if (!enc) return false;
    const cuuint32_t group = (cuuint32_t)(p.num_q_heads / p.num_kv_heads);
    cuuint64_t dims[3] = {(cuuint64_t)p.head_dim, (cuuint64_t)p.num_q_heads, (cuuint64_t)p.num_seqs};
    cuuint64_t strides[2] = {(cuuint64_t)p.head_dim * 2, (cuuint64_t)p.num_q_heads * p.head_dim * 2};
    cuuint32_t box[3] = {64, group, 32 / group};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p.q), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Steps of the longest list: every group at its largest, every prefix at its longest.
int64_t most_steps(const pa_decode_shared_params &p) {
    const int64_t group = p.dec.num_q_heads / p.dec.num_kv_heads;
    const int64_t per = item_rows(p.dec.kv_dtype), tiles = ((int64_t)p.max_group * group + per - 1) / per;
    const int64_t steps = ((int64_t)p.max_prefix + kBN - 1) / kBN;
    return p.num_groups * tiles * (steps + kItemSteps) * p.dec.num_kv_heads;
}

int most_ctas(const pa_decode_shared_params &p) {
    const int64_t steps = most_steps(p), sms = num_sms();
    return (int)(steps < sms ? steps : sms);
}

// Measured, of a step: 3200 clocks for two tiles of head size 128, 5000 where rows are
// gathered one by one, 1260 to 1600 over FP8 at 64, 1950 over 4 bits at 128.  The split-KV
// decode reads 38 GB/s an SM.  One figure per type of pool: other head sizes and groups of
// a single tile are not measured; a figure that is off costs time only.
void set_costs(SharedArgs &sh, const pa_decode_shared_params &p) {
    const pa_decode_params &d = p.dec;
    const float bytes = d.kv_dtype == PA_KV_BF16 ? 4.f : d.kv_dtype == PA_KV_FP4 ? 1.125f : 2.f;     // of an element, K and V
    sh.sms = num_sms();
    sh.step_ns = d.page_size == 1 ? 2600.f : d.kv_dtype == PA_KV_BF16 ? 1700.f : d.kv_dtype == PA_KV_FP4 ? 1000.f : 700.f;
    sh.key_ns = bytes * (float)(d.head_dim * d.num_kv_heads) / 38.f;
}

// The prefix kernel's grid beside a tail: at least 3/4 of the SMs, and what is best for
// the call's bounds.  The kernel may leave more of them (shared_ctas), 4 us later.
unsigned prefix_ctas(const pa_decode_shared_params &p, const SharedArgs &sh) {
    const int all = most_ctas(p);
    if (p.max_suffix == 0 || all < sh.sms) return (unsigned)all;
    const float steps = (float)most_steps(p) * sh.step_ns;
    const float rest = shared_rest(sh, (float)p.dec.num_seqs * (float)p.max_suffix, p.dec.num_kv_heads);
    int best = all;
    for (int i = 31; i >= 24; --i) {
        const int n = all * i / 32;
        if (shared_time(steps, rest, n, sh.sms) < shared_time(steps, rest, best, sh.sms)) best = n;
    }
    return (unsigned)best;
}

}  // namespace

// The decode call over the keys behind the prefixes.  In a 4-bit pool they may
// begin and end inside a unit of 16 keys.
pa_decode_params shared_tail_params(const pa_decode_shared_params &p) {
    pa_decode_params d = p.dec;
    d.max_seqlen_k = p.max_suffix + (p.dec.kv_dtype == PA_KV_FP4 && p.max_suffix > 0 ? 16 : 0);
    return d;
}

// At least the workspace of any split-KV decode of up to num_seqs sequences of up to
// max_seqlen_k keys: automatic ranges have 64 keys or more, and 1/32 of the longest
// sequence or more, so that a shorter bound may need more than this one.
static size_t split_workspace_any(const pa_decode_params &d, const DecodePlan &plan) {
    if (d.kv_dtype == PA_KV_FP4 || d.kv_chunk != 0) return plan.workspace_any;
    const int64_t by_keys = ((int64_t)d.max_seqlen_k + 63) / 64 + 1;
    const size_t slots = (size_t)d.num_seqs * d.num_q_heads * (by_keys < 33 ? by_keys : 33);
    return 256 + round256(((size_t)d.num_seqs + 1) * sizeof(int32_t)) + round256(slots * d.head_dim * sizeof(float)) +
           slots * sizeof(float);
}

SharedPlan plan_decode_shared(const pa_decode_shared_params &p) {
    SharedPlan plan{};
    plan.prefix = p.num_groups > 0 && p.max_prefix > 0 && p.max_group > 0 && p.dec.num_seqs > 0;
    plan.tail = p.max_suffix > 0;
    if (plan.prefix) {
        // an item for each range and row of the list, less one (prefill_impl.cuh); a
        // row for every KV head and item_rows query rows of a group, or part of them
        const int64_t group = p.dec.num_q_heads / p.dec.num_kv_heads;
        const int64_t per = item_rows(p.dec.kv_dtype);
        const int64_t whole = (int64_t)p.dec.num_seqs * group / per + p.num_groups;
        const int64_t bound = p.num_groups * (((int64_t)p.max_group * group + per - 1) / per);
        plan.max_blocks = (int32_t)(most_ctas(p) + (whole < bound ? whole : bound) * p.dec.num_kv_heads);
        const size_t rows = (size_t)plan.max_blocks * kBlockRows;
        plan.prefix_bytes = 256 + 256 + round256((size_t)p.num_groups * sizeof(int2)) + rows * p.dec.head_dim * sizeof(float) +
                            rows * sizeof(float);
    }
    const pa_decode_params tail = shared_tail_params(p);
    if (plan.tail) {
        plan.decode = tail.kv_dtype == PA_KV_FP4 ? plan_decode_fp4(tail) : plan_decode(tail);
        plan.decode.workspace_any = split_workspace_any(tail, plan.decode);
    }
    plan.workspace_bytes = plan.prefix_bytes + plan.decode.workspace_any;
    if (plan.workspace_bytes < 256) plan.workspace_bytes = 256;
    // (a call without groups decodes every key as pa_decode does)
    const size_t whole = split_workspace_any(p.dec, p.dec.kv_dtype == PA_KV_FP4 ? plan_decode_fp4(p.dec) : plan_decode(p.dec));
    plan.workspace_any = whole > plan.workspace_bytes ? whole : plan.workspace_bytes;
    return plan;
}

cudaError_t launch_decode_shared(const pa_decode_shared_params &p, const SharedPlan &plan, cudaStream_t stream) {
    const pa_decode_params &d = p.dec;
    MergeArgs m{};
    m.sh.cu_groups = p.cu_groups;
    m.sh.prefix_lens = p.prefix_lens;
    m.sh.num_groups = p.num_groups;
    m.sh.max_group = p.max_group;
    m.sh.max_prefix = plan.prefix ? p.max_prefix : 0;
    m.sh.max_blocks = plan.max_blocks;
    set_costs(m.sh, p);
    if (plan.tail) {
        m.sh.cache_seqlens = d.cache_seqlens;
        m.sh.max_suffix = p.max_suffix;
    }
    // (the partials are stored 32 bytes at a time)
    uint8_t *ws = reinterpret_cast<uint8_t *>(round256(reinterpret_cast<uintptr_t>(d.workspace)));
    if (plan.prefix) {
        const size_t rows = (size_t)plan.max_blocks * kBlockRows;
        uint8_t *o = ws + 256 + round256((size_t)p.num_groups * sizeof(int2));
        m.sh.header = reinterpret_cast<int32_t *>(ws);
        m.sh.base = reinterpret_cast<int2 *>(ws + 256);
        m.sh.o_part = reinterpret_cast<float *>(o);
        m.sh.lse_part = reinterpret_cast<float *>(o + rows * d.head_dim * sizeof(float));
        PrefillArgs a{};
        const int64_t num_slots = d.num_pages * d.page_size;
        if (!make_map_shared_q(&a.qmap, d)) return cudaErrorNotSupported;
        if (d.kv_dtype == PA_KV_FP4) a.lay = fp4_layout(d.num_kv_heads, d.head_dim);
        if (d.page_size == 16) {
            for (int i = 0; i < 2; ++i) {
                CUtensorMap *map = i == 0 ? &a.kmap : &a.vmap;
                const void *pool = i == 0 ? d.k_cache : d.v_cache;
                const bool ok = d.kv_dtype == PA_KV_FP4 ? make_map_fp4(map, pool, a.lay.row_bytes, num_slots, d.head_dim / 2)
                                : d.kv_dtype == PA_KV_FP8_E4M3 ? make_map_fp8(map, pool, d.head_dim, d.num_kv_heads, num_slots, 16)
                                                               : make_map(map, pool, d.head_dim, d.num_kv_heads, num_slots, 16);
                if (!ok) return cudaErrorNotSupported;
            }
        }
        a.k_cache = static_cast<const uint8_t *>(d.k_cache);
        a.v_cache = static_cast<const uint8_t *>(d.v_cache);
        a.page_table = d.page_table;
        a.pt_stride = d.page_table_stride;
        a.num_seqs = d.num_seqs;
        a.num_q_heads = d.num_q_heads;
        a.num_kv_heads = d.num_kv_heads;
        a.page_size = d.page_size;
        a.num_slots = (int32_t)num_slots;
        a.scale_log2 = d.scale * 1.4426950408889634f;
        a.k_scale = d.k_scale;
        a.v_scale = d.v_scale;
        a.sh = m.sh;
        const unsigned ctas = prefix_ctas(p, m.sh);
        const cudaError_t e = d.kv_dtype == PA_KV_FP4        ? launch_prefix<PA_KV_FP4>(a, d.head_dim, ctas, stream)
                              : d.kv_dtype == PA_KV_FP8_E4M3 ? launch_prefix<PA_KV_FP8_E4M3>(a, d.head_dim, ctas, stream)
                                                             : launch_prefix<PA_KV_BF16>(a, d.head_dim, ctas, stream);
        if (e != cudaSuccess) return e;
    }
    if (plan.tail) {
        // Its CTAs start as the prefix kernel's leave the SMs; it reads nothing of
        // that kernel's, which has waited for all that came before.
        pa_decode_params t = d;
        t.workspace = static_cast<uint8_t *>(d.workspace) + plan.prefix_bytes;
        t.workspace_bytes = d.workspace_bytes - plan.prefix_bytes;
        t.overlap_previous = plan.prefix ? 1 : 0;
        m.tail.first_keys = p.prefix_lens;
        m.tail.max_keys = p.max_suffix;
        const cudaError_t e = d.kv_dtype == PA_KV_FP4 ? launch_decode_fp4(t, plan.decode, stream, &m.tail)
                                                      : launch_decode(t, plan.decode, stream, &m.tail);
        if (e != cudaSuccess) return e;
    }
    m.cache_seqlens = d.cache_seqlens;
    m.num_seqs = d.num_seqs;
    m.num_q_heads = d.num_q_heads;
    m.num_kv_heads = d.num_kv_heads;
    m.max_seqlen_k = d.max_seqlen_k;
    m.item_rows = item_rows(d.kv_dtype);
    m.out = static_cast<__nv_bfloat16 *>(d.out);
    m.lse = d.lse;
    return launch_merge(m, d.head_dim, stream);
}

}  // namespace pa
