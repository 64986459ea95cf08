// LayerNorm kernels with fp16 activations: the instantiations of layernorm_impl.cuh.
#include "layernorm_impl.cuh"

namespace rmsn {

cudaError_t layernorm_f16_read_error(unsigned* flags, bool clear) { return read_ln_error_word(flags, clear); }
cudaError_t launch_ln_fwd_f16(const LnFwdArgs& a, cudaStream_t s) { return ln_fwd_dispatch<true>(a, s); }
cudaError_t launch_ln_bwd_f16(const LnBwdArgs& a, unsigned chunks, bool bias, cudaStream_t s) {
    return bias ? ln_bwd_dispatch<true, true>(a, chunks, s) : ln_bwd_dispatch<true, false>(a, chunks, s);
}

}  // namespace rmsn
