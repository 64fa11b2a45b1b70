// Windowed / paged tcgen05 chunked-prefill instantiations with 2-bit keys
// (single-width values at 1..4 bits, and the fractional-rate caches: keys 2/1,
// values 2/1, 3/2, 4/3 code bits) and an fp32 output.
#include "prefill_view.cuh"

namespace tqk {

cudaError_t launch_prefill_view_k2_f32(const PrefillParams& p, int vbits, bool two, cudaStream_t s) {
    return prefill_view_k2<true>(p, vbits, two, s);
}

}  // namespace tqk
