// The head norm fused with rotary positions, backward, bf16 activations: the
// instantiations of rope_impl.cuh.
#include "rope_impl.cuh"

namespace rmsn {

cudaError_t rope_norm_bwd_read_error(unsigned* flags, bool clear) { return read_rope_error_word(flags, clear); }
cudaError_t launch_rope_norm_bwd(const RopeArgs& a, int* ctas_q, cudaStream_t s) { return rope_kinds<kNormTurnBwd, false>(a, ctas_q, s); }

}  // namespace rmsn
