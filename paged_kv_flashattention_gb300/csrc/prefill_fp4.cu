// Varlen causal prefill / extend attention over 4-bit pools: the instantiations
// of prefill_impl.cuh that widen E2M1 tiles, and their launch.
#include "prefill_impl.cuh"

namespace pa {

PA_ERROR_WORD_ACCESSOR(error_word_prefill_fp4)

namespace {

template <int D, int T, bool EXT>
__global__ void __launch_bounds__(128 * (T + 1), 1) prefill_fp4_kernel(const __grid_constant__ PrefillArgs a) {
    prefill_body<D, T, true, EXT, true>(a);
}

template <int D, int T, bool EXT>
cudaError_t launch_t(const PrefillArgs &a, unsigned ctas, cudaStream_t stream) {
    using S = PrefillSmem<D, T, true, true>;
    static_assert(S::kSlots >= 3 && S::kCSlots >= 3, "ring too small");
    static_assert(S::kTotal + 1024 <= 232448, "shared memory");
    // One CTA per SM (it allocates all 512 TMEM columns).
    const int smem = (S::kTotal + 1024) > 120 * 1024 ? (S::kTotal + 1024) : 120 * 1024;
    auto kern = prefill_fp4_kernel<D, T, EXT>;
    if (T == 2) {
        static const cudaError_t regs = check_register_split(kern);
        if (regs != cudaSuccess) return regs;
    }
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kern<<<ctas, 128 * (T + 1), smem, stream>>>(a);
    return cudaGetLastError();
}

template <bool EXT>
cudaError_t dispatch(const PrefillArgs &a, int d, int T, unsigned ctas, cudaStream_t stream) {
    if (d == 128) return T == 2 ? launch_t<128, 2, EXT>(a, ctas, stream) : launch_t<128, 1, EXT>(a, ctas, stream);
    return T == 2 ? launch_t<64, 2, EXT>(a, ctas, stream) : launch_t<64, 1, EXT>(a, ctas, stream);
}

}  // namespace

cudaError_t launch_prefill_fp4(const pa_prefill_params &p, cudaStream_t stream) {
    PrefillArgs a;
    int T = 1;
    cudaError_t e = prefill_setup(p, a, T);
    if (e != cudaSuccess) return e;
    if (a.num_virtual == 0) return cudaSuccess;
    a.sched = p.scheduler;
    int64_t ctas = num_sms();
    if (p.max_ctas > 0 && p.max_ctas < ctas) ctas = p.max_ctas;
    if (a.num_virtual < ctas) ctas = a.num_virtual;
    a.num_ctas = (int32_t)ctas;
    return (a.window > 0 || a.bmask != nullptr) ? dispatch<true>(a, p.head_dim, T, (unsigned)ctas, stream)
                                                : dispatch<false>(a, p.head_dim, T, (unsigned)ctas, stream);
}

}  // namespace pa
