// Windowed / paged tcgen05 chunked-prefill instantiations with 1-bit keys and a
// bf16 output; fp32 outputs and 2-bit keys in prefill_view_f32.cu,
// prefill_view2.cu and prefill_view2_f32.cu.
#include "prefill_view.cuh"

namespace tqk {

cudaError_t launch_prefill_view_k1_f32(const PrefillParams& p, int vbits, cudaStream_t s);
cudaError_t launch_prefill_view_k2(const PrefillParams& p, int vbits, bool two, cudaStream_t s);
cudaError_t launch_prefill_view_k2_f32(const PrefillParams& p, int vbits, bool two, cudaStream_t s);

cudaError_t launch_prefill_umma_view(const PrefillParams& p, int kbits, int vbits, bool two, bool f32_out, cudaStream_t s) {
    if (p.chunk <= 0 || p.batch <= 0 || p.n_splits <= 0) return cudaSuccess;
    if (!prefill_umma_supported(kbits, vbits, two)) return cudaErrorInvalidValue;
    if (kbits == 2) return f32_out ? launch_prefill_view_k2_f32(p, vbits, two, s) : launch_prefill_view_k2(p, vbits, two, s);
    return f32_out ? launch_prefill_view_k1_f32(p, vbits, s) : prefill_view_k1<false>(p, vbits, s);
}

}  // namespace tqk
