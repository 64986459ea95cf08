// Internal launch interface of the projections' kernels between their C-ABI layer
// (linear.cu) and the translation units with the kernels. Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "linear.h"

namespace rmsn {

// A 16-bit matrix by its first value and its row stride in elements.
struct MatIn { const uint16_t* p; int64_t ld; };
struct MatOut { uint16_t* p; int64_t ld; };

// What a product's epilogue does with the accumulators.
enum ProductKind : int {
    kForward = 0,  // out = round(act(acc + b) + res), z = round(acc + b);   C = A B^T
    kGatedFwd = 1, // out = round(act(acc0) * acc1), z, z2 = round(acc0), round(acc1); C = A B^T of two B
    kGradX = 2,    // out = round(acc);                                       C = A B, of one or two pairs
    kGradW = 3     // out = round(acc) or, split, fp32 sums of its rows' range; C = A^T B, of one or two A
};

// C [M][N], summed over K. The operands as they lie in memory:
//   kForward, kGatedFwd: A [M][K], B [N][K];  kGradX: A [M][K], B [K][N];  kGradW: A [K][M], B [K][N].
// Second operands: kGatedFwd b[1]; kGradX a[1], b[1] (a second product added); kGradW a[1] (a second output).
struct Product {
    MatIn a[2], b[2];
    MatOut out[2];
    MatOut z[2];         // kept pre-activations (p null: not kept)
    MatIn res;
    const float* bias;
    float* partials;     // kGradW, splits > 1: [output][split][M][N]
    int64_t M, N, K;
    int splits;
    int act;
};

cudaError_t launch_linear_fwd(ProductKind kind, const Product& p, cudaStream_t s);
cudaError_t launch_linear_fwd_f16(ProductKind kind, const Product& p, cudaStream_t s);
cudaError_t launch_linear_grad(ProductKind kind, const Product& p, cudaStream_t s);
cudaError_t launch_linear_grad_f16(ProductKind kind, const Product& p, cudaStream_t s);

// The gradients of the activations: dz = g act'(z) (out[0]; null: not written) and, if
// `partials` is not null, its columns' sums over `ranges` ranges of rows. With `up`
// (gated): dgate = g up act'(z) (out[0]), dup = g act(z) (out[1]).
struct Slopes {
    MatIn g, z, up;
    MatOut out[2];
    float* partials;  // [ranges][N]
    int64_t T, N, ranges;
    int act;
};
cudaError_t launch_linear_slopes(const Slopes& a, bool f16, cudaStream_t s);
// out = round(sum of `splits` partials [M][N], in order)
cudaError_t launch_linear_join(const float* partials, int splits, const MatOut& out, int64_t M, int64_t N, bool f16,
                               cudaStream_t s);

cudaError_t linear_fwd_read_error(unsigned* flags, bool clear);
cudaError_t linear_fwd_f16_read_error(unsigned* flags, bool clear);
cudaError_t linear_grad_read_error(unsigned* flags, bool clear);
cudaError_t linear_grad_f16_read_error(unsigned* flags, bool clear);

}  // namespace rmsn
