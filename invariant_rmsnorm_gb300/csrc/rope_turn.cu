// Rotary positions alone, bf16 activations: the
// instantiations of rope_impl.cuh.
#include "rope_impl.cuh"

namespace rmsn {

cudaError_t rope_turn_read_error(unsigned* flags, bool clear) { return read_rope_error_word(flags, clear); }
cudaError_t launch_rope_turn(const RopeArgs& a, int* ctas_q, cudaStream_t s) { return rope_kinds<kTurn, false>(a, ctas_q, s); }

}  // namespace rmsn
