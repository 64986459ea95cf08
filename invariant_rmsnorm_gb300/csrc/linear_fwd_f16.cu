// Projections and gated blocks forward, fp16 values: the instantiations of linear_impl.cuh.
#include "linear_impl.cuh"

namespace rmsn {

cudaError_t linear_fwd_f16_read_error(unsigned* flags, bool clear) { return read_linear_error_word(flags, clear); }
cudaError_t launch_linear_fwd_f16(ProductKind kind, const Product& p, cudaStream_t s) {
    return kind == kGatedFwd ? product_shape<kGatedFwd, true>(p, s) : product_shape<kForward, true>(p, s);
}

}  // namespace rmsn
