// Windowed / paged tcgen05 chunked-prefill instantiations with 1-bit keys and an
// fp32 output.
#include "prefill_view.cuh"

namespace tqk {

cudaError_t launch_prefill_view_k1_f32(const PrefillParams& p, int vbits, cudaStream_t s) {
    return prefill_view_k1<true>(p, vbits, s);
}

}  // namespace tqk
