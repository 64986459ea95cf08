// Gradients of the projections' inputs and weights, fp16 values: the instantiations of linear_impl.cuh.
#include "linear_impl.cuh"

namespace rmsn {

cudaError_t linear_grad_f16_read_error(unsigned* flags, bool clear) { return read_linear_error_word(flags, clear); }
cudaError_t launch_linear_grad_f16(ProductKind kind, const Product& p, cudaStream_t s) {
    return kind == kGradX ? product_shape<kGradX, true>(p, s) : product_shape<kGradW, true>(p, s);
}

}  // namespace rmsn
