// Gradients of the projections' inputs and weights, bf16 values: the instantiations of linear_impl.cuh.
#include "linear_impl.cuh"

namespace rmsn {

cudaError_t linear_grad_read_error(unsigned* flags, bool clear) { return read_linear_error_word(flags, clear); }
cudaError_t launch_linear_grad(ProductKind kind, const Product& p, cudaStream_t s) {
    return kind == kGradX ? product_shape<kGradX, false>(p, s) : product_shape<kGradW, false>(p, s);
}

}  // namespace rmsn
