// Rotary positions of several axes, fp16 activations: the
// instantiations of rope_impl.cuh.
#include "rope_impl.cuh"

namespace rmsn {

cudaError_t rope_axes_turn_f16_read_error(unsigned* flags, bool clear) { return read_rope_error_word(flags, clear); }
cudaError_t launch_rope_axes_turn_f16(const RopeArgs& a, int* ctas_q, cudaStream_t s) {
    return rope_kinds<kTurn, true, true>(a, ctas_q, s);
}

}  // namespace rmsn
