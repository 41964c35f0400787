// The batch's metadata from request lengths that live on the device: the
// boundaries of "code-series sgl-project mini-sglang 07" ("from ledger to
// tensors": cached_len, extend_len, device_len = cached_len + extend_len), the
// new tokens' positions and slots, the page table, and (optionally) the pages
// that the new tokens need, taken from a free list and entered in the
// token-granular table.
//
// With e_b = extend_len, c_b = cached_len, P = page_size:
//   cu_q = prefix(e), cu_k = prefix(c + e), pages_b = ceil((c_b + e_b) / P),
//   new_b = pages_b - ceil(c_b / P), first_b = prefix(new)
//   token i of request b: position p = c_b + i; its page is the one its last
//   cached token lies on while p / P < ceil(c_b / P), else
//   free_pages[first_b + p / P - ceil(c_b / P)]; slot = page * P + p % P.
// Every output element depends on the lengths through three prefix sums alone,
// so there is one launch and no hand-over between CTAs: each CTA forms the
// sums in shared memory (at most 16384 requests, 12 bytes each) and then takes
// its share of the tokens and of the page-table entries, finding an element's
// request by bisection.  Entries of the token table are read below c_b and
// written from c_b on, so the order of the two does not matter.
//
// With a cursor (pa_build_batch_from) the list starts at free_pages[cursor[0]].
// Every CTA reads that before it counts itself in cursor[1]; the CTA that counts
// last moves cursor[0] past the pages taken and clears cursor[1], so nothing
// waits and the next launch in the stream finds both ready.
// Bound: launch latency and the CTA's chain (two dependent passes over L2, three
// prefix sums, 64-bit divisions per request and element) for a decode step (256
// requests 7.5 us), the token table's 32-byte sectors (one per page at page size
// 16), the bisections and the lengths read again per element for large tables
// (1000 requests of up to 8408 keys, 253,000 new tokens 9.6 us).
#include "pa_device.cuh"
#include "pa_internal.h"
#include "pdl.cuh"

namespace pa {

PA_ERROR_WORD_ACCESSOR(error_word_batch)

namespace {

// Two CTAs of 512 threads per SM: 9.6 us on the 1000 requests; four of 256 12.5,
// one of 1024 10.5, four of 512 11.4 (every CTA forms the prefixes).
constexpr int kThreads = 512;
constexpr int kCtasPerSm = 2;

struct Lens {
    int cached, extend;           // 0, 0 for a request whose lengths break the call's bounds
    int row;                      // row of the token table; -1 outside it
};

__device__ __forceinline__ Lens request(const pa_batch_params &p, int b) {
    Lens r{p.cached_len[b], p.extend_len[b], p.table_idx[b]};
    if (r.cached < 0 || r.extend < 0 || (int64_t)r.cached + r.extend > p.max_seqlen_k) r.cached = r.extend = 0;
    if (r.row < 0 || r.row >= p.token_table_rows) r.row = -1;
    return r;
}

__device__ __forceinline__ int pages_of(int keys, int P) { return (int)(((int64_t)keys + P - 1) / P); }

// a[0] = 0, a[1 .. n] become their running sums; every thread of the CTA.
__device__ void running_sum(int32_t *a, int n, int32_t *warp_sums) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int per = (n + kThreads - 1) / kThreads;
    const int from = 1 + t * per, to = min(n, t * per + per);
    int run = 0;
    for (int i = from; i <= to; ++i) run += a[i];
    int incl = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int acc = incl - run;
    for (int w = 0; w < warp; ++w) acc += warp_sums[w];
    for (int i = from; i <= to; ++i) {
        acc += a[i];
        a[i] = acc;
    }
    __syncthreads();
}

// The request whose range [a[b], a[b+1]) holds i.
__device__ __forceinline__ int find(const int32_t *a, int n, int i) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= i) lo = mid; else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int floor_div(int x, int P) {
    int q = x / P;
    if (x < 0 && q * P != x) --q;
    return q;
}

// The page of new page number n of the batch; -1 once the list, from entry
// `from` on, is used up.
__device__ __forceinline__ int free_page(const pa_batch_params &p, int from, int n) {
    if (n < p.num_free_pages - from) return p.free_pages[from + n];
    raise_error(PA_DEVERR_NO_PAGES);
    return -1;
}

__global__ void __launch_bounds__(kThreads) build_batch_kernel(const pa_batch_params p, int32_t *cursor) {
    extern __shared__ int32_t smem[];
    __shared__ int32_t warp_sums[kThreads / 32];
    __shared__ int32_t list_from;
    after_previous();
    const int B = p.num_seqs, P = p.page_size;
    const bool take = p.free_pages != nullptr;
    if (threadIdx.x == 0) {                          // (a cursor outside the list: a list that is used up)
        const int at = cursor != nullptr ? *reinterpret_cast<volatile int32_t *>(cursor) : 0;
        list_from = at < 0 || at > p.num_free_pages ? p.num_free_pages : at;
    }
    int32_t *cq = smem;                              // [B + 1] new tokens
    int32_t *cp = cq + B + 1;                        // [B + 1] pages
    int32_t *cn = cp + B + 1;                        // [B + 1] pages to take
    for (int b = threadIdx.x; b < B; b += kThreads) {
        const Lens r = request(p, b);
        cq[b + 1] = r.extend;
        cp[b + 1] = pages_of(r.cached + r.extend, P);
        cn[b + 1] = take && r.row >= 0 ? pages_of(r.cached + r.extend, P) - pages_of(r.cached, P) : 0;
    }
    if (threadIdx.x == 0) cq[0] = cp[0] = cn[0] = 0;
    __syncthreads();
    running_sum(cq, B, warp_sums);
    running_sum(cp, B, warp_sums);
    if (take) running_sum(cn, B, warp_sums);
    const int total = cq[B], pages = cp[B];
    const int from = list_from;                      // (read after the barriers above)
    if (cursor != nullptr && threadIdx.x == 0) {
        __threadfence();                             // this CTA's read of cursor[0] before its count
        if (atomicAdd(&cursor[1], 1) == (int)gridDim.x - 1) {
            cursor[0] = from + min(cn[B], p.num_free_pages - from);
            cursor[1] = 0;
        }
    }

    const int64_t stride = (int64_t)gridDim.x * kThreads;
    const int64_t me = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    for (int64_t t = me; t < p.num_tokens; t += stride) {
        int pos = 0, slot = -1;                      // entries past the batch's tokens
        if (t < total) {
            const int b = find(cq, B, (int)t);
            const Lens r = request(p, b);
            pos = r.cached + (int)t - cq[b];
            if (r.row >= 0) {
                int32_t *row = p.token_table + r.row * p.token_table_stride;
                if (take) {
                    const int fresh = pos / P - pages_of(r.cached, P);
                    const int page = fresh >= 0 ? free_page(p, from, cn[b] + fresh) : floor_div(row[r.cached - 1], P);
                    slot = page >= 0 ? page * P + pos % P : -1;
                    row[pos] = slot;
                } else {
                    slot = row[pos];
                }
            }
        }
        p.positions[t] = pos;
        p.slot_mapping[t] = slot;
    }
    for (int64_t i = me; i < pages; i += stride) {
        const int b = find(cp, B, (int)i), c = (int)i - cp[b];
        const Lens r = request(p, b);
        int page = -1;
        if (r.row >= 0) {
            const int fresh = c - pages_of(r.cached, P);
            page = take && fresh >= 0 ? free_page(p, from, cn[b] + fresh)
                                      : floor_div(p.token_table[r.row * p.token_table_stride + (int64_t)c * P], P);
        }
        p.page_table[(int64_t)b * p.page_table_stride + c] = page;
    }

    if (blockIdx.x != 0) return;
    for (int b = threadIdx.x; b <= B; b += kThreads) p.cu_seqlens_q[b] = cq[b];
    __syncthreads();
    int most_q = 0, most_k = 0;
    for (int b = threadIdx.x; b < B; b += kThreads) {
        const Lens r = request(p, b);
        cp[b + 1] = r.cached + r.extend;
        p.cache_seqlens[b] = r.cached + r.extend;
        most_q = max(most_q, r.extend);
        most_k = max(most_k, r.cached + r.extend);
        const int c = p.cached_len[b], e = p.extend_len[b];
        if (c < 0 || e < 0 || (int64_t)c + e > p.max_seqlen_k) raise_error(PA_DEVERR_SEQLENS);
        if (r.row < 0) raise_error(PA_DEVERR_TABLE_INDEX);
    }
    __syncthreads();
    running_sum(cp, B, warp_sums);
    for (int b = threadIdx.x; b <= B; b += kThreads) p.cu_seqlens_k[b] = cp[b];
    __shared__ int32_t most[2];
    if (threadIdx.x < 2) most[threadIdx.x] = 0;
    __syncthreads();
    atomicMax(&most[0], most_q);
    atomicMax(&most[1], most_k);
    __syncthreads();
    if (threadIdx.x == 0) {
        if (total > p.num_tokens) raise_error(PA_DEVERR_SEQLENS);
        p.totals[0] = total;
        p.totals[1] = most[0];
        p.totals[2] = most[1];
        p.totals[3] = cn[B];
    }
}

}  // namespace

cudaError_t launch_build_batch(const pa_batch_params &p, int32_t *free_cursor, cudaStream_t stream) {
    const size_t smem = 3 * ((size_t)p.num_seqs + 1) * sizeof(int32_t);
    if (smem > 40 * 1024) {                          // more than a CTA has without asking (with the static part)
        cudaError_t e = cudaFuncSetAttribute(build_batch_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
        if (e != cudaSuccess) return e;
    }
    const int64_t cols = ((int64_t)p.max_seqlen_k + p.page_size - 1) / p.page_size;
    int64_t blocks = (p.num_tokens + cols * p.num_seqs + kThreads - 1) / kThreads;
    const int64_t cap = (int64_t)num_sms() * kCtasPerSm;
    if (blocks > cap) blocks = cap;
    if (blocks < 1) blocks = 1;
    return launch_after(build_batch_kernel, (unsigned)blocks, kThreads, smem, stream, p, free_cursor);
}

}  // namespace pa
