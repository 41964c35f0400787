// Beam search over a paged cache: the selection over beams and vocabulary, and
// the reordering of the paged states that follows it.
//
// Selection.  total[k, v] = score[k] + x[k, v] - lse[k], the n largest of a
// group's beams * V totals.  Within a row the order is that of x, so one pass
// over the logits finds each chunk's n largest and its part of lse; a second
// launch, one CTA per group, forms lse and the totals in 64 bits and merges the
// chunks' lists.
//   - A CTA has a threshold that n of its elements reach: the n-th largest of its
//     thread maxima.  Elements above it go to a buffer in shared memory (little more
//     than n), all others into the sum of exponentials at once, with the threshold as
//     reference: it bounds them.  A buffer that fills up is cut to its n largest.  An
//     entry's rank among the buffer's is its place in the list.
//   - Finding the threshold, ranking and 64-bit exponentials take a CTA 5 us,
//     whatever it has read.  Small calls read a chunk into registers and pay that
//     once; large ones stream the logits by (maximum, sum) of 32 columns, and a CTA
//     per row reads the few blocks again that hold its n largest.
//   - Two candidates of different beams are ordered by sums that differ by lse, so the
//     n largest exponentials are summed in 64 bits, and the rest, each off by about
//     2^-22 of itself, in 32 per thread over a few hundred elements and then in 64.
//     Measured against 64 bits (128256 logits; normal with deviations of 0.01 to 6,
//     of eight values, with one peak; bf16 and fp32), lse is off by up to 4e-8 where a
//     call takes chunks and 1.2e-7 where it takes two passes.  Most of it is ex2's own
//     and one-sided: with log2 e in two parts the second is 1.7e-7, since the rounded
//     one happens to lean the other way.  In 64 groups of totals about 0.05 apart,
//     neighbours of different beams swap once in several hundred steps.
//   - Columns belong to threads by their number, whatever the row's alignment,
//     so that equal rows give equal sums and their ties go by index.
//
// Reordering.  Rows of the partly filled last pages are one contiguous run of a
// page, copied into the child's spare page first (CTAs of one sequence and a few
// pools each); a second launch, beside it, permutes the token-table rows and
// histories, a thread per column, which holds the column's values of all beams.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pdl.cuh"

namespace pa {

PA_ERROR_WORD_ACCESSOR(error_word_beam)

namespace {

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kElems = 8;                            // columns of a thread in a tile
constexpr int kTile = kSelThreads * kElems;
constexpr int kKept = 512;                           // entries that stay in the buffer between tiles
constexpr float kLog2e = 1.4426950408889634f;

struct ChunkSum {
    double top;                   // the chunk's largest logit (-inf: no finite one)
    double sum;                   // sum of exp(x - top)
};

struct SelectArgs {
    const void *logits;
    int64_t stride;
    const float *scores;
    const uint8_t *finished;
    int32_t pad, groups, beams, vocab, n;
    int32_t chunks;               // lists of a row
    int32_t spans;                // CTAs of a row in the first pass of large calls
    float2 *lists;                // [rows][chunks][n]: logit, column as bits (0xffffffff: none)
    ChunkSum *sums;               // [rows][chunks]
    float2 *blocks;               // [rows][spans][kSelThreads]: maximum, sum
    float *out_scores;
    int32_t *out_parents;
    int32_t *out_tokens;
    uint8_t *out_finished;
};

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t ai = *reinterpret_cast<uint64_t *>(&a), bi = *reinterpret_cast<uint64_t *>(&b), r;
    asm("add.f32x2 %0, %1, %2;" : "=l"(r) : "l"(ai), "l"(bi));
    return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t ai = *reinterpret_cast<uint64_t *>(&a), bi = *reinterpret_cast<uint64_t *>(&b), r;
    asm("mul.f32x2 %0, %1, %2;" : "=l"(r) : "l"(ai), "l"(bi));
    return *reinterpret_cast<float2 *>(&r);
}

// Scores that are no numbers count as -inf.
__device__ __forceinline__ float cleaned(float x) { return x < INFINITY ? x : -INFINITY; }

__device__ __forceinline__ bool beam_reads(const SelectArgs &a, int row) {
    return !(a.finished != nullptr && a.finished[row] != 0) && cleaned(a.scores[row]) != -INFINITY;
}

// Floats as unsigned words in the same order; -0 as 0.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
// A larger logit, then a smaller column, gives a larger key.
__device__ __forceinline__ uint64_t key_of(float x, int col) { return (uint64_t)ordered(x) << 32 | (uint32_t)~col; }
__device__ __forceinline__ float key_value(uint64_t k) { return unordered((uint32_t)(k >> 32)); }

template <int DT>
__device__ __forceinline__ float element(const void *row, int64_t i) {
    if constexpr (DT == PA_LOGITS_F32) return static_cast<const float *>(row)[i];
    else if constexpr (DT == PA_LOGITS_F16) return __half2float(static_cast<const __half *>(row)[i]);
    else return __bfloat162float(static_cast<const __nv_bfloat16 *>(row)[i]);
}

// kElems columns as loaded: whole 16-byte words that begin `skew` bytes before the
// first column, or (skew 0 then) single elements.
template <int DT>
struct Columns {
    static constexpr int kBytes = DT == PA_LOGITS_F32 ? 4 : 2;
    static constexpr int kWords = kElems * kBytes / 4;
    uint32_t w[kWords + 4];
    bool whole;

    // Columns col .. of a row that ends at `end`, -inf behind it.  Words are read
    // only if they end inside the row.
    __device__ __forceinline__ void load(const uint8_t *row, int skew, int col, int end) {
        whole = col + kElems + (skew != 0 ? 16 / kBytes : 0) <= end;
        if (whole) {
            const uint4 *p = reinterpret_cast<const uint4 *>(row + (int64_t)col * kBytes - skew);
#pragma unroll
            for (int i = 0; i < kWords / 4 + 1; ++i) {
                if (i == kWords / 4 && skew == 0) break;
                const uint4 v = p[i];
                w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
            }
        } else {
            uint32_t e[kElems];
#pragma unroll
            for (int i = 0; i < kElems; ++i) {
                const bool in = col + i < end;
                if constexpr (kBytes == 4) e[i] = in ? reinterpret_cast<const uint32_t *>(row)[col + i] : 0xff800000u;
                else e[i] = in ? reinterpret_cast<const uint16_t *>(row)[col + i] : DT == PA_LOGITS_F16 ? 0xfc00u : 0xff80u;
            }
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = kBytes == 4 ? e[i] : e[2 * i] | e[2 * i + 1] << 16;
        }
    }

    // Moves the first column to the first word.
    __device__ __forceinline__ void align(int skew) {
        if (whole && skew != 0) {                    // (the same for all whole threads of a row)
            if (skew & 8)
#pragma unroll
                for (int i = 0; i < kWords + 2; ++i) w[i] = w[i + 2];
            if (skew & 4)
#pragma unroll
                for (int i = 0; i < kWords + 1; ++i) w[i] = w[i + 1];
            if (skew & 2)
#pragma unroll
                for (int i = 0; i < kWords; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
        }
    }

    __device__ __forceinline__ void values(float (&x)[kElems]) const {
#pragma unroll
        for (int i = 0; i < kElems; ++i) {
            if constexpr (DT == PA_LOGITS_F32) {
                x[i] = __uint_as_float(w[i]);
            } else if constexpr (DT == PA_LOGITS_BF16) {
                x[i] = (i & 1) ? bf16hi(w[i / 2]) : bf16lo(w[i / 2]);
            } else {
                const __half2 h = *reinterpret_cast<const __half2 *>(&w[i / 2]);
                x[i] = (i & 1) ? __high2float(h) : __low2float(h);
            }
        }
    }
};

// A value that n of the CTA's thread maxima reach and few others do: their n-th
// largest with the bits below `low` cleared (0 is below all values).  One warp
// finds it bit by bit, 16 bits in about 700 clocks; the least of the warps'
// (n / warps)-th largest would take 100, but lets through three times as many
// elements, and all of a tile of which one warp has none.
__device__ __forceinline__ uint32_t block_floor(uint32_t top, int n, int low, uint32_t (&tops)[kSelThreads]) {
    const int lane = threadIdx.x & 31;
    tops[threadIdx.x] = top;
    __syncthreads();
    if (threadIdx.x < 32) {
        uint32_t v[kSelWarps];
#pragma unroll
        for (int i = 0; i < kSelWarps; ++i) v[i] = tops[lane + 32 * i];
        uint32_t at = 0;
        for (int bit = 31; bit >= low; --bit) {
            const uint32_t trial = at | 1u << bit;
            uint32_t reach = 0;
#pragma unroll
            for (int i = 0; i < kSelWarps; ++i) reach += v[i] >= trial;
            if ((int)__reduce_add_sync(0xffffffffu, reach) >= n) at = trial;
        }
        __syncwarp();
        if (lane == 0) tops[0] = at;
    }
    __syncthreads();
    return tops[0];
}

// The largest value below an ordered word's (-0 is 0).
__device__ __forceinline__ float value_below(uint32_t k) { return unordered(k - 1 == 0x7fffffffu ? k - 2 : k - 1); }

// A buffer is cut when it holds more than this; it then has room for another tile
// (round), every element of which may be an entry.
__device__ __forceinline__ int kept_limit(int n) { return 16 + n + n / 2; }

// A CTA's n largest of the elements that it is shown, and the sum of all of their
// exponentials.  Elements above the threshold are entries of the buffer; the others
// are in `rest`, each thread's sum of 2^((x - ref) log2 e) with ref = thr, its value.
struct Chosen {
    uint64_t buf[kKept + kTile];
    uint64_t best[128];
    uint32_t tops[kSelThreads];
    unsigned long long dropped;                      // in units of 2^-32: of the buffer, until thread 0 takes it
    unsigned long long whole;                        // in the same units: all threads' rest, once they are through
    int count;
};

struct Chooser {
    Chosen &sh;
    int n, limit;
    float thr, ref, rest;
    // Keys above this one, whose value is thr, are due.  Where columns come in their order
    // nothing behind a cut of value thr is, and the values alone tell.
    uint64_t floor;

    __device__ __forceinline__ Chooser(Chosen &s, int n)
        : sh(s), n(n), limit(kept_limit(n)), thr(-INFINITY), ref(0.f), rest(0.f), floor(key_of(-INFINITY, 0)) {
        if (threadIdx.x == 0) {
            sh.count = 0;
            sh.dropped = 0;
            sh.whole = 0;
        }
    }
    __device__ __forceinline__ float term(float x) const { return fast_exp2((x - ref) * kLog2e); }
    // A new threshold, the same for the CTA.
    __device__ __forceinline__ void raise(float to, uint64_t key) {
        const float r = to == -INFINITY ? 0.f : to;
        rest = rest > 0.f ? rest * fast_exp2((ref - r) * kLog2e) : 0.f;
        thr = to;
        ref = r;
        floor = key;
    }
    // The first threshold, from the maxima of the threads' elements: elements of
    // that value are entries too.
    __device__ __forceinline__ void start(float most) {
        const uint32_t least = block_floor(ordered(most), n, 16, sh.tops);
        if (least > ordered(-INFINITY)) raise(value_below(least), key_of(value_below(least), 0));
    }
    // An element above thr, or of a key above floor; the entries then (they may be more than the limit).
    __device__ __forceinline__ int enter(float x, int col) {
        const int at = atomicAdd(&sh.count, 1);
        sh.buf[at] = key_of(x, col);
        return at + 1;
    }
    // Cuts the buffer's m entries to the n largest, in order, in best; the n-th is
    // the new threshold and the others go into rest: as whole multiples of 2^-32, so
    // that their order in the buffer, which is chance, does not matter.  Every thread.
    __device__ int cut(int m) {
        const int t = threadIdx.x;
        uint32_t out = 0;
        for (int e = t, i = 0; e < m; e += kSelThreads, ++i) {
            const uint64_t k = sh.buf[e];
            int rank = 0;
#pragma unroll 8
            for (int j = 0; j < m; ++j) rank += sh.buf[j] > k;
            if (rank < n) sh.best[rank] = k;
            else out |= 1u << i;
        }
        __syncthreads();
        if (m < n) return m;
        raise(key_value(sh.best[n - 1]), sh.best[n - 1]);
        if (out != 0) {
            unsigned long long sum = 0;
            for (int e = t, i = 0; e < m; e += kSelThreads, ++i)
                if (out >> i & 1u) sum += (unsigned long long)__float2ull_rn(term(key_value(sh.buf[e])) * 0x1p32f);
            atomicAdd(&sh.dropped, sum);
        }
        __syncthreads();
        if (t == 0) {
            rest += (float)sh.dropped * 0x1p-32f;
            sh.dropped = 0;
        }
        return n;
    }
    // Between batches of at most kTile elements: room for the next.  `last` is the
    // thread's last enter().
    __device__ __forceinline__ void settle(int last) {
        if (__syncthreads_or(last > limit)) {
            const int kept = cut(sh.count);          // limit >= n: n entries stay
            if ((int)threadIdx.x < kept) sh.buf[threadIdx.x] = sh.best[threadIdx.x];
            if (threadIdx.x == 0) sh.count = kept;
            __syncthreads();
        }
    }
    // The list, and the sum with the list's exponentials in 64 bits; returns the
    // list's length.
    __device__ int finish(float2 *list, ChunkSum *to) {
        const int lane = threadIdx.x & 31;
        __syncthreads();
        const int kept = cut(sh.count);
        // rest of all threads, each to 2^-32 of the least term of the list, in whole
        // numbers of two halves.  Not in `dropped`: thread 0 may not have cleared that.
        const unsigned long long units = __float2ull_rn(rest * 0x1p32f);
        const uint32_t lo = __reduce_add_sync(0xffffffffu, (uint32_t)units & 0xffffffu);
        const uint32_t hi = __reduce_add_sync(0xffffffffu, (uint32_t)(units >> 24));
        if (lane == 0) atomicAdd(&sh.whole, ((unsigned long long)hi << 24) + lo);
        __syncthreads();
        const float top = kept > 0 ? key_value(sh.best[0]) : -INFINITY;
        if (threadIdx.x < 32) {
            double sum = 0.0;
            for (int e = lane; e <= kept; e += 32) { // entry `kept`: the rest, at its reference
                const float x = e < kept ? key_value(sh.best[e]) : ref;
                if (e < kept) list[e] = make_float2(x, __int_as_float((int)~(uint32_t)sh.best[e]));
                if (e < kept || sh.whole != 0)
                    sum += exp((double)x - (double)top) * (e < kept ? 1.0 : (double)sh.whole * 0x1p-32);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) *to = ChunkSum{(double)top, sum};
        }
        return kept;
    }
};

// Fills a list of `kept` entries up to n with the first columns of [from, end) that
// are -inf, and to a.n with none.  Warp 0.
template <int DT>
__device__ void fill_list(float2 *list, int kept, int n, int most, const uint8_t *row, int from, int end) {
    const int lane = threadIdx.x & 31;
    int have = kept;
    for (int col = from; col < end && have < n; col += 32) {
        const bool none = col + lane < end && cleaned(element<DT>(row, col + lane)) == -INFINITY;
        const unsigned who = __ballot_sync(0xffffffffu, none);
        const int place = have + __popc(who & ((1u << lane) - 1u));
        if (none && place < n) list[place] = make_float2(-INFINITY, __int_as_float(col + lane));
        have += __popc(who);
    }
    for (int e = n + lane; e < most; e += 32) list[e] = make_float2(-INFINITY, __uint_as_float(0xffffffffu));
}

__device__ __forceinline__ float max_of(const float (&x)[kElems]) {      // the larger of numbers
    float top = x[0];
#pragma unroll
    for (int i = 1; i < kElems; ++i) top = fmaxf(top, x[i]);
    return top;
}
__device__ __forceinline__ float sum_of(const float (&x)[kElems]) {
    float2 s = make_float2(x[0], x[1]);
#pragma unroll
    for (int i = 2; i < kElems; i += 2) s = add2(s, make_float2(x[i], x[i + 1]));
    return s.x + s.y;
}
__device__ __forceinline__ void terms_of(const float (&x)[kElems], float ref, float (&e)[kElems]) {
#pragma unroll
    for (int i = 0; i < kElems; i += 2) {
        const float2 y = mul2(add2(make_float2(x[i], x[i + 1]), make_float2(-ref, -ref)), make_float2(kLog2e, kLog2e));
        e[i] = fast_exp2(y.x);
        e[i + 1] = fast_exp2(y.y);
    }
}

// Small calls: a CTA's chunk of U tiles in registers, its maxima first: the
// threshold is then one that little more than n of its elements reach.
template <int DT, int U>
__global__ void __launch_bounds__(kSelThreads) select_chunks_kernel(const SelectArgs a) {
    __shared__ Chosen shared;
    after_previous();
    const int t = threadIdx.x;
    const int row_id = blockIdx.x / a.chunks, c = blockIdx.x % a.chunks;
    if (!beam_reads(a, row_id)) return;
    constexpr int kBytes = DT == PA_LOGITS_F32 ? 4 : 2;
    const uint8_t *row = static_cast<const uint8_t *>(a.logits) + (int64_t)row_id * a.stride * kBytes;
    const int skew = (int)(reinterpret_cast<uintptr_t>(row) & 15u);
    const int from = c * (U * kTile), end = min(from + U * kTile, a.vocab);
    Chooser ch(shared, min(a.n, end - from));
    Columns<DT> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u].load(row, skew, from + u * kTile + t * kElems, end);
    float tops_of[U], most = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float x[kElems];
        raw[u].align(skew);
        raw[u].values(x);
        tops_of[u] = max_of(x);
        if (tops_of[u] == INFINITY) {
#pragma unroll
            for (int i = 0; i < kElems; ++i) most = fmaxf(most, cleaned(x[i]));
        } else {
            most = fmaxf(most, tops_of[u]);
        }
    }
    ch.start(most);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float x[kElems], e[kElems];
        const int col = from + u * kTile + t * kElems;
        raw[u].values(x);
        // Most warps have no element above the threshold: they add their terms and are
        // done.  (A maximum leaves NaN out, the sum of the terms does not; +inf is above
        // every threshold.)
        int last = 0;
        terms_of(x, ch.ref, e);
        float terms = sum_of(e);
        if (__any_sync(0xffffffffu, tops_of[u] > ch.thr || !(terms < INFINITY))) {
            uint32_t above = 0;
#pragma unroll
            for (int i = 0; i < kElems; ++i) {
                const float v = cleaned(x[i]);
                if (v > ch.thr) above |= 1u << i;
                // a term that is no number: its element is not one either
                e[i] = v > ch.thr || !(v > -INFINITY) ? 0.f : e[i];
            }
            terms = sum_of(e);
            while (above != 0u) {
                const int i = __ffs(above) - 1;
                above &= above - 1u;
                float v = x[0];
#pragma unroll
                for (int q = 1; q < kElems; ++q) v = i == q ? x[q] : v;
                last = ch.enter(v, col + i);
            }
        }
        if (ch.thr != -INFINITY) ch.rest += terms;
        ch.settle(last);
    }
    const int64_t at = (int64_t)row_id * a.chunks + c;
    float2 *list = a.lists + at * a.n;
    const int kept = ch.finish(list, a.sums + at);
    if (kept < a.n && t < 32) fill_list<DT>(list, kept, ch.n, a.n, row, from, end);
}

// Large calls, first pass: of every thread's kBlockTiles x 8 columns their maximum
// and the sum of exp(x - maximum), nothing else, so that the logits stream through.
constexpr int kBlockTiles = 4;
constexpr int kSpan = kBlockTiles * kTile;           // columns of a CTA

template <int DT>
__global__ void __launch_bounds__(kSelThreads) select_blocks_kernel(const SelectArgs a) {
    after_previous();
    const int t = threadIdx.x;
    const int row_id = blockIdx.x / a.spans, c = blockIdx.x % a.spans;
    if (a.finished != nullptr && !beam_reads(a, row_id)) return;
    constexpr int kBytes = DT == PA_LOGITS_F32 ? 4 : 2;
    const uint8_t *row = static_cast<const uint8_t *>(a.logits) + (int64_t)row_id * a.stride * kBytes;
    const int skew = (int)(reinterpret_cast<uintptr_t>(row) & 15u);
    const int from = c * kSpan + t * kElems;
    Columns<DT> raw[kBlockTiles];
#pragma unroll
    for (int u = 0; u < kBlockTiles; ++u) raw[u].load(row, skew, from + u * kTile, a.vocab);
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < kBlockTiles; ++u) {
        float x[kElems];
        raw[u].align(skew);
        raw[u].values(x);
        top = fmaxf(top, max_of(x));
    }
    float sum = 0.f;
#pragma unroll
    for (int u = 0; u < kBlockTiles; ++u) {
        float x[kElems], e[kElems];
        raw[u].values(x);
        terms_of(x, top, e);
        sum += sum_of(e);
    }
    if (!(sum < INFINITY)) {                         // NaN or +inf among them, or nothing but -inf
        top = -INFINITY;
        sum = 0.f;
#pragma unroll
        for (int u = 0; u < kBlockTiles; ++u) {
            float x[kElems];
            raw[u].values(x);
#pragma unroll
            for (int i = 0; i < kElems; ++i) top = fmaxf(top, cleaned(x[i]));
        }
        if (top > -INFINITY) {
#pragma unroll
            for (int u = 0; u < kBlockTiles; ++u) {
                float x[kElems];
                raw[u].values(x);
#pragma unroll
                for (int i = 0; i < kElems; ++i) sum += fast_exp2((cleaned(x[i]) - top) * kLog2e);
            }
        }
    }
    a.blocks[((int64_t)row_id * a.spans + c) * kSelThreads + t] = make_float2(top, sum);
}

// Second pass, a CTA per row: the n-th largest of the threads' maxima over the
// blocks is the threshold; only blocks that reach it (little more than n) are read
// again, of the others their sums count.  Blocks are listed in their order, so that
// the sums do not depend on chance.  A block's columns lie in four tiles, so a
// smaller column may come behind a larger one: what is due behind a cut is told by
// whole keys, of equal values the smaller columns.
constexpr int kListed = 1024;

template <int DT>
__global__ void __launch_bounds__(kSelThreads) select_rows_kernel(const SelectArgs a) {
    __shared__ Chosen shared;
    __shared__ int list_of[kListed], found[kListed], warp_count[kSelWarps], total;
    after_previous();
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, row_id = blockIdx.x;
    if (!beam_reads(a, row_id)) return;
    constexpr int kBytes = DT == PA_LOGITS_F32 ? 4 : 2;
    const uint8_t *row = static_cast<const uint8_t *>(a.logits) + (int64_t)row_id * a.stride * kBytes;
    const float2 *blocks = a.blocks + (int64_t)row_id * a.spans * kSelThreads;
    Chooser ch(shared, a.n);
    float most = -INFINITY;
#pragma unroll 8
    for (int c = 0; c < a.spans; ++c) most = fmaxf(most, blocks[c * kSelThreads + t].x);
    ch.start(most);
    auto read_again = [&](int listed) {              // 32 blocks a batch, 8 threads a block, a thread 4 x 1 columns
        for (int base = 0; base < listed; base += 32) {
            const int mine = base + (t >> 3);
            int last = 0;
            if (mine < listed) {
                const int id = list_of[mine];
                const int first = id / kSelThreads * kSpan + id % kSelThreads * kElems, col0 = first + (t & 7);
                float v[kBlockTiles];
#pragma unroll
                for (int u = 0; u < kBlockTiles; ++u)
                    v[u] = col0 + u * kTile < a.vocab ? cleaned(element<DT>(row, col0 + u * kTile)) : -INFINITY;
                const float2 b = blocks[id];
                if (key_of(b.x, first) > ch.floor) { // (no key of the block is larger)
#pragma unroll
                    for (int u = 0; u < kBlockTiles; ++u) {
                        if (key_of(v[u], col0 + u * kTile) > ch.floor) last = ch.enter(v[u], col0 + u * kTile);
                        else if (v[u] > -INFINITY) ch.rest += ch.term(v[u]);
                    }
                } else if ((t & 7) == 0) {           // the threshold has passed it since
                    ch.rest += b.y * ch.term(b.x);
                }
            }
            ch.settle(last);
        }
    };
    if (t == 0) total = 0;
    __syncthreads();
#pragma unroll 8
    for (int c = 0; c < a.spans; ++c) {
        const float2 b = blocks[c * kSelThreads + t];
        if (b.x > ch.thr) {
            const int at = atomicAdd(&total, 1);
            if (at < kListed) found[at] = c * kSelThreads + t;
        } else if (b.y > 0.f) {
            ch.rest += b.y * ch.term(b.x);
        }
    }
    __syncthreads();
    if (total <= kListed) {                          // in the order of their numbers
        const int m = total;
        for (int e = t; e < m; e += kSelThreads) {
            const int id = found[e];
            int rank = 0;
            for (int i = 0; i < m; ++i) rank += found[i] < id;
            list_of[rank] = id;
        }
        __syncthreads();
        read_again(m);
    } else {                                         // rows of equal logits: kSelThreads blocks at a time
        const float first = ch.thr;
        for (int c = 0; c < a.spans; ++c) {
            const bool again = blocks[c * kSelThreads + t].x > first;
            const unsigned who = __ballot_sync(0xffffffffu, again);
            if (lane == 0) warp_count[warp] = __popc(who);
            __syncthreads();
            int at = __popc(who & ((1u << lane) - 1u)), listed = 0;
#pragma unroll
            for (int w = 0; w < kSelWarps; ++w) {
                if (w < warp) at += warp_count[w];
                listed += warp_count[w];
            }
            if (again) list_of[at] = c * kSelThreads + t;
            __syncthreads();
            read_again(listed);
        }
    }
    float2 *list = a.lists + (int64_t)row_id * a.n;
    const int kept = ch.finish(list, a.sums + row_id);
    if (kept < a.n && t < 32) fill_list<DT>(list, kept, ch.n, a.n, row, 0, a.vocab);
}

// One CTA per group: lse of its beams, the totals of the lists' entries, the n
// largest of those.  lse is kept as the largest logit and the logarithm of the sum:
// in one number a row of the type's lowest value would lose the logarithm.  Entries pass the threshold in rounds, as above; beams whose
// logits are not read offer what they have in place of their first list.
constexpr int kRound = 4 * kSelThreads;
constexpr int kBuf2 = kKept + kRound;

// Doubles as unsigned words in the same order; -0 as 0.
__device__ __forceinline__ uint64_t ordered(double x) {
    const uint64_t b = (uint64_t)__double_as_longlong(x + 0.0);
    return (b >> 63) ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ double unordered(uint64_t k) {
    return __longlong_as_double((long long)((k >> 63) ? k & ~(1ull << 63) : ~k));
}

__global__ void __launch_bounds__(kSelThreads) select_merge_kernel(const SelectArgs a) {
    __shared__ uint64_t tot[kBuf2], best_tot[128];
    __shared__ uint32_t idx[kBuf2], best_idx[128], tops[kSelThreads];
    __shared__ double tops_of[64], logs[64];         // lse of a beam = their sum
    __shared__ float score[64];
    __shared__ uint8_t state[64];                    // 0: reads its logits, 1: ended, 2: score -inf
    __shared__ uint8_t flags[64];                    // finished, read before any of it may be overwritten
    __shared__ int count;
    after_previous();
    const int t = threadIdx.x, lane = t & 31, g = blockIdx.x;
    const int K = a.beams, S = a.chunks, n = a.n, limit = kept_limit(n);
    if (t == 0) count = 0;
    for (int k = t >> 5; k < K; k += kSelWarps) {    // a warp per beam: its state, its lse
        const float s = cleaned(a.scores[g * K + k]);
        const uint8_t flag = a.finished != nullptr ? a.finished[g * K + k] : 0;
        const int st = s == -INFINITY ? 2 : flag != 0 ? 1 : 0;
        double top = -INFINITY, l = 0.0;
        if (st == 0) {
            const ChunkSum *cs = a.sums + ((int64_t)g * K + k) * S;
            double sum = 0.0;
            for (int c = lane; c < S; c += 32) top = fmax(top, cs[c].top);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (top > -INFINITY)
                for (int c = lane; c < S; c += 32) sum += cs[c].sum * (cs[c].top == top ? 1.0 : exp(cs[c].top - top));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            l = log(sum);                            // (no finite logit: not used)
        }
        if (lane == 0) {
            score[k] = s;
            state[k] = (uint8_t)st;
            flags[k] = flag;
            tops_of[k] = top;
            logs[k] = l;
        }
    }
    __syncthreads();

    const unsigned per_beam = (unsigned)(S * n), entries = (unsigned)K * per_beam;
    // Entry e's ordered total, 0 for none, and its beam and column.
    auto entry = [&](unsigned e, uint32_t &at) -> uint64_t {
        const int k = (int)(e / per_beam), r = (int)(e % per_beam);
        at = 0xffffffffu;
        if (state[k] == 0) {
            const float2 x = a.lists[((int64_t)g * K + k) * per_beam + r];
            const uint32_t col = __float_as_uint(x.y);
            if (col == 0xffffffffu) return 0;
            at = (uint32_t)k << 24 | col;
            return ordered(x.x == -INFINITY ? (double)-INFINITY : (double)score[k] + (((double)x.x - tops_of[k]) - logs[k]));
        }
        if (r >= n) return 0;                        // n <= vocab columns
        int col = r;
        if (state[k] == 1) col = r == 0 ? a.pad : r - 1 + (r - 1 >= a.pad);
        at = (uint32_t)k << 24 | (uint32_t)col;
        return ordered(state[k] == 1 && r == 0 ? (double)score[k] : (double)-INFINITY);
    };
    uint64_t thr = 0;                                // with thr_idx: the n-th best so far
    uint32_t thr_idx = 0xffffffffu, least = 0;       // least: n entries of the first round have as much
    auto better = [](uint64_t x, uint32_t i, uint64_t y, uint32_t j) { return x > y || (x == y && i < j); };
    // Ranks the buffer's m entries; the n best, in order, into best.
    auto cut = [&](int m) {
        for (int e = t; e < m; e += kSelThreads) {
            const uint64_t v = tot[e];
            const uint32_t at = idx[e];
            int rank = 0;
#pragma unroll 4
            for (int i = 0; i < m; ++i) rank += better(tot[i], idx[i], v, at);
            if (rank < n) {
                best_tot[rank] = v;
                best_idx[rank] = at;
            }
        }
        __syncthreads();
        return min(m, n);
    };
    for (unsigned e0 = 0; e0 < entries; e0 += kRound) {
        uint64_t v[kRound / kSelThreads];
        uint32_t at[kRound / kSelThreads];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kRound / kSelThreads; ++i) {
            const unsigned e = e0 + i * kSelThreads + t;
            v[i] = 0;
            at[i] = 0xffffffffu;
            if (e < entries) v[i] = entry(e, at[i]);
            top = max(top, (uint32_t)(v[i] >> 32));
        }
        if (e0 == 0 && entries > 128) least = block_floor(top, n, 12, tops);
        int last = 0;
#pragma unroll
        for (int i = 0; i < kRound / kSelThreads; ++i) {
            if (v[i] == 0 || (uint32_t)(v[i] >> 32) < least || !better(v[i], at[i], thr, thr_idx)) continue;
            last = atomicAdd(&count, 1);
            tot[last] = v[i];
            idx[last] = at[i];
            ++last;
        }
        if (__syncthreads_or(last > limit)) {
            const int kept = cut(count);
            if (t < kept) {
                tot[t] = best_tot[t];
                idx[t] = best_idx[t];
            }
            if (t == 0) count = kept;
            __syncthreads();
            if (kept == n) {
                thr = best_tot[n - 1];
                thr_idx = best_idx[n - 1];
            }
        }
    }
    __syncthreads();
    cut(count);
    for (int e = t; e < n; e += kSelThreads) {
        const uint32_t at = best_idx[e];
        a.out_scores[(int64_t)g * n + e] = (float)unordered(best_tot[e]);
        a.out_parents[(int64_t)g * n + e] = (int)(at >> 24);
        a.out_tokens[(int64_t)g * n + e] = (int)(at & 0xffffffu);
        if (a.out_finished != nullptr) a.out_finished[(int64_t)g * n + e] = flags[at >> 24];
    }
}

// ------------------------------------------------------------- reordering ---
struct ReorderArgs {
    pa_beam_reorder_params p;
    void *pools[PA_BEAM_REORDER_MAX_POOLS];
};

// Length of group g's sequences, -1 if they differ or break the bounds (every
// thread of the CTA, the answer for all).
__device__ __forceinline__ int group_length(const pa_beam_reorder_params &p, int g) {
    const int32_t *lens = p.seqlens + (int64_t)g * p.beams;
    const int L = lens[0];
    bool bad = L < 0 || L > p.max_seqlen_k;
    for (int k = threadIdx.x; k < p.beams; k += blockDim.x) bad |= lens[k] != L;
    return __syncthreads_or(bad) ? -1 : L;
}

__device__ __forceinline__ bool row_ok(const pa_beam_reorder_params &p, int row) { return row >= 0 && row < p.token_table_rows; }

// The parent of beam i of group g if it moves, else i itself.
__device__ __forceinline__ int parent_of(const pa_beam_reorder_params &p, int g, int i) {
    const int64_t base = (int64_t)g * p.beams;
    const int q = p.parents[base + i];
    if (q == i) return i;
    if (q < 0 || q >= p.beams || !row_ok(p, p.table_idx[base + i]) || !row_ok(p, p.table_idx[base + q])) {
        raise_error(PA_DEVERR_TABLE_INDEX);
        return i;
    }
    return q;
}

constexpr int kCopyThreads = 256;

// CTA (sequence, slice of the pools): the rows of the parent's last page into the
// sequence's spare page.
__global__ void __launch_bounds__(kCopyThreads) reorder_copy_kernel(const __grid_constant__ ReorderArgs a, int slices) {
    const pa_beam_reorder_params &p = a.p;
    after_previous();
    const int seq = blockIdx.x / slices, slice = blockIdx.x % slices;
    const int g = seq / p.beams, i = seq % p.beams;
    const int parent = p.parents[seq];
    if (parent == i) return;
    const int L = group_length(p, g);
    const int part = L % p.page_size;
    if (L <= 0 || part == 0) return;
    const int q = parent_of(p, g, i);
    if (q == i) return;
    const int32_t slot = p.token_table[p.table_idx[(int64_t)g * p.beams + q] * p.token_table_stride + L - 1];
    const int32_t src = slot >= 0 ? slot / p.page_size : -1, dst = p.spare_pages[seq];
    // Every thread has read what the next launch overwrites: it may start beside the copies.
    const bool bad = __syncthreads_or(src < 0 || src >= p.num_pages || dst < 0 || dst >= p.num_pages);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (bad) {
        if (threadIdx.x == 0) raise_error(PA_DEVERR_PAGE_RANGE);
        return;
    }
    const int64_t page_words = p.row_bytes / 16 * p.page_size;
    const int words = (int)(p.row_bytes / 16 * part);
    for (int k = slice; k < p.num_pools; k += slices) {
        uint4 *pool = static_cast<uint4 *>(a.pools[k]);
        const uint4 *from = pool + src * page_words;
        uint4 *to = pool + dst * page_words;
        constexpr int U = 8;
        for (int w0 = threadIdx.x; w0 < words; w0 += U * kCopyThreads) {
            uint4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (w0 + u * kCopyThreads < words) v[u] = from[w0 + u * kCopyThreads];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (w0 + u * kCopyThreads < words) to[w0 + u * kCopyThreads] = v[u];
        }
    }
}

constexpr int kColumns = 128;                        // columns of a CTA, a multiple of every page size

// CTA (group, block of columns): first the token table's blocks, then the
// histories'.  The CTA of a group's last slots also turns the spare pages over.
__device__ __forceinline__ void reorder_rows(const pa_beam_reorder_params &p, int table_blocks, int blocks) {
    extern __shared__ int32_t vals[];                // [beams][kColumns], each thread its own column
    __shared__ int parents[64], spares[64], firsts[64];
    __shared__ int64_t rows[64];                     // a row's first cell, -1 outside the table
    const int g = blockIdx.x / blocks, block = blockIdx.x % blocks, t = threadIdx.x;
    const int64_t base = (int64_t)g * p.beams;
    const bool table = block < table_blocks;
    const int col = (table ? block : block - table_blocks) * kColumns + t;
    const int L = group_length(p, g);
    if (L < 0) {
        if (t == 0) raise_error(PA_DEVERR_SEQLENS);
        return;
    }
    const int part = L % p.page_size, full = L - part;       // slots from `full` on lie on the last page
    const int ends = table ? L : p.history_len;
    if (col - t >= ends) return;
    const bool last = table && part > 0 && col - t + kColumns >= L;
    bool moves = false;
    for (int k = t; k < p.beams; k += kColumns) {
        const int q = parent_of(p, g, k);
        const int idx = p.table_idx[base + k];
        parents[k] = q;
        rows[k] = !table ? (base + k) * p.history_stride : row_ok(p, idx) ? idx * p.token_table_stride : -1;
        firsts[k] = table && p.prefix_lens != nullptr ? p.prefix_lens[base + k] : 0;
        spares[k] = last ? p.spare_pages[base + k] : -1;
        moves |= q != k && (last || col - t + kColumns > firsts[k]);
    }
    if (!__syncthreads_or(moves) || col >= ends) return;
    int32_t *cells = table ? p.token_table : p.history;
    for (int k = 0; k < p.beams; ++k)
        if (rows[k] >= 0) vals[k * kColumns + t] = cells[rows[k] + col];
    for (int k = 0; k < p.beams; ++k) {
        const int q = parents[k];
        if (q == k) continue;                        // (else both rows are in the table)
        int32_t *cell = cells + rows[k] + col;
        if (table && col >= full) {
            const int32_t own = vals[k * kColumns + t];
            *cell = spares[k] >= 0 && spares[k] < p.num_pages ? spares[k] * p.page_size + col - full : -1;
            if (col == L - 1) p.spare_pages[base + k] = own >= 0 ? own / p.page_size : -1;
        } else if (col >= firsts[k]) {
            *cell = vals[q * kColumns + t];
        }
    }
}

// after_copies: the launch before is the copies', which has waited for all before it
// and let this one start once its CTAs had read the table and the spare pages.  The
// last CTA ends after the copies, and with it the grid.
__global__ void __launch_bounds__(kColumns) reorder_rows_kernel(const pa_beam_reorder_params p, int table_blocks, int blocks,
                                                                bool after_copies) {
    if (!after_copies) after_previous();
    reorder_rows(p, table_blocks, blocks);
    if (after_copies && blockIdx.x == gridDim.x - 1) after_previous();
}

constexpr int kMostTiles = 4;     // tiles of a chunk where there are CTAs enough
constexpr int kSmallTiles = 3000; // tiles of a call whose chunks are not worth a pass of their own

template <int DT>
cudaError_t launch_lists(const SelectArgs &a, int tiles, cudaStream_t stream) {
    const unsigned rows = (unsigned)(a.groups * a.beams);
    if (tiles > 0)
        return launch_after(tiles == 1 ? select_chunks_kernel<DT, 1> : select_chunks_kernel<DT, kMostTiles>, rows * a.chunks,
                            kSelThreads, 0, stream, a);
    const cudaError_t e = launch_after(select_blocks_kernel<DT>, rows * a.spans, kSelThreads, 0, stream, a);
    return e != cudaSuccess ? e : launch_after(select_rows_kernel<DT>, rows, kSelThreads, 0, stream, a);
}

size_t round16(size_t n) { return (n + 15) / 16 * 16; }

}  // namespace

// Calls of up to kSmallTiles tiles: a list per chunk of kMostTiles tiles, or of one
// while the GPU holds all CTAs at once; larger ones: a list per row by two passes.
// (Constant numbers: the workspace's size is the same on every device.)
// A smaller call may have more lists than a larger one, so the size reported is the
// largest of any with as many rows, tiles and entries or fewer: r rows of t tiles have
// r t lists for r t <= kOneTile, then at most r ceil(t / kMostTiles) <= r t, then r.
SelectPlan plan_select(const pa_beam_select_params &p) {
    constexpr int64_t kOneTile = 152 * 4;
    SelectPlan plan{};
    const int64_t rows = (int64_t)p.num_groups * p.beams, tiles = ((int64_t)p.vocab + kTile - 1) / kTile;
    plan.tiles = rows * tiles <= kOneTile ? 1 : rows * tiles <= kSmallTiles ? kMostTiles : 0;
    plan.chunks = plan.tiles > 0 ? (int32_t)((tiles + plan.tiles - 1) / plan.tiles) : 1;
    plan.spans = (int32_t)((tiles + kBlockTiles - 1) / kBlockTiles);
    auto list_bytes = [&](int64_t lists) { return round16((size_t)lists * p.num_out * sizeof(float2)); };
    auto sum_bytes = [&](int64_t lists) { return round16((size_t)lists * sizeof(ChunkSum)); };
    plan.list_bytes = list_bytes(rows * plan.chunks);
    plan.sum_bytes = sum_bytes(rows * plan.chunks);
    plan.workspace_bytes = plan.list_bytes + plan.sum_bytes;
    if (plan.tiles == 0) plan.workspace_bytes += (size_t)rows * plan.spans * kSelThreads * sizeof(float2);
    int64_t lists = std::min(rows * tiles, kOneTile);
    if (rows * tiles > kOneTile)
        lists = std::max(lists, std::min(rows * ((tiles + kMostTiles - 1) / kMostTiles), (int64_t)kSmallTiles));
    plan.workspace_any = std::max(plan.workspace_bytes, list_bytes(lists) + sum_bytes(lists));
    return plan;
}

cudaError_t launch_select(const pa_beam_select_params &p, const SelectPlan &plan, cudaStream_t stream) {
    SelectArgs a{};
    a.logits = p.logits;
    a.stride = p.logits_stride;
    a.scores = p.scores;
    a.finished = p.finished;
    a.pad = p.pad_token;
    a.groups = p.num_groups;
    a.beams = p.beams;
    a.vocab = p.vocab;
    a.n = p.num_out;
    a.chunks = plan.chunks;
    a.spans = plan.spans;
    uint8_t *ws = static_cast<uint8_t *>(p.workspace);
    a.lists = reinterpret_cast<float2 *>(ws);
    a.sums = reinterpret_cast<ChunkSum *>(ws + plan.list_bytes);
    a.blocks = reinterpret_cast<float2 *>(ws + plan.list_bytes + plan.sum_bytes);
    a.out_scores = p.out_scores;
    a.out_parents = p.out_parents;
    a.out_tokens = p.out_tokens;
    a.out_finished = p.out_finished;
    const cudaError_t e = p.logits_dtype == PA_LOGITS_F32   ? launch_lists<PA_LOGITS_F32>(a, plan.tiles, stream)
                          : p.logits_dtype == PA_LOGITS_F16 ? launch_lists<PA_LOGITS_F16>(a, plan.tiles, stream)
                                                            : launch_lists<PA_LOGITS_BF16>(a, plan.tiles, stream);
    if (e != cudaSuccess) return e;
    return launch_after(select_merge_kernel, (unsigned)p.num_groups, kSelThreads, 0, stream, a);
}

cudaError_t launch_reorder(const pa_beam_reorder_params &p, cudaStream_t stream) {
    const int seqs = p.num_groups * p.beams;
    const bool copies = p.page_size > 1 && p.num_pools > 0;
    if (copies) {
        ReorderArgs a{};
        a.p = p;
        for (int k = 0; k < p.num_pools; ++k) a.pools[k] = p.pools[k];
        // a few CTAs for every SM; a CTA finds its pages once for its pools
        int slices = (num_sms() * 8 + seqs - 1) / seqs;
        if (slices > p.num_pools) slices = p.num_pools;
        const cudaError_t e = launch_after(reorder_copy_kernel, (unsigned)(seqs * slices), kCopyThreads, 0, stream, a, slices);
        if (e != cudaSuccess) return e;
    }
    const int table_blocks = (p.max_seqlen_k + kColumns - 1) / kColumns;
    const int blocks = table_blocks + (p.history != nullptr ? (p.history_len + kColumns - 1) / kColumns : 0);
    if (blocks == 0) return cudaSuccess;
    pa_beam_reorder_params q = p;
    if (q.history == nullptr) q.history_len = 0;
    return launch_after(reorder_rows_kernel, (unsigned)((int64_t)p.num_groups * blocks), kColumns,
                        (size_t)p.beams * kColumns * sizeof(int32_t), stream, q, table_blocks, blocks, copies);
}

}  // namespace pa
