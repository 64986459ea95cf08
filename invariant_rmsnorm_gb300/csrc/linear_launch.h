// Internal launch interface of the projections' kernels between their C-ABI layer
// (linear.cu) and the translation units with the kernels. Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

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

// A product's tile: CTAs (two: a pair, 256 rows), rows a CTA, columns of accumulators, and the model's cycles.
struct Tiling { int ctas, rows, bn; int64_t cycles; };

constexpr int kMostDeep = 8, kMostDeepPair = 2;      // blocks of 64 reduced values a stage
constexpr uint32_t kStageBytes = 227 * 1024 - 2048;  // of shared memory for the stages

// The tile by a model of a GPU of 152 SMs, in cycles. Tiles go round it in waves, of 76 pairs or
// 152 single CTAs. A block of a tile takes a pair of 256 x 256 512 (its products) and of 256 x 128 270
// (290 with both operands along their columns) in a single wave, 340 (390) in more: its operands are three quarters
// of the larger tile's for half the products (8192 x 4096 x 16384: 796 us for 666); a single CTA its products, 2 a
// column, or their operands from shared memory, 1 a row and column, or from L2 at 80 bytes a cycle, or 140 and 310
// a stage of the issuing thread; a tile at least its epilogue, 12 a column; a launch of pairs 900 more. Single CTAs
// have as many columns as give every SM one tile or, past 256, two and more (a multiple of 16; of 32 with two
// matrices' columns, of 64 where B lies along them), and 64 rows up to 64 in all, 64 or 128 beyond.
// Where rows of the operands do not start on lines (`lines` false) their way is 45 bytes a cycle and SM: 2048 x 4104 x 4096
// 697 cycles a block of 256 x 256 and 521 of 256 x 128.
// 512 x 4096 x 4096: pairs of 256 x 128 13.6 us, single CTAs of 128 columns 18.1; 1024 x 4096 x 4096: 20.8 and,
// with 256 x 256, 23.0; 64 x 4096 x 6144: CTAs of 48 columns 12.3, of 64 13.1; 128 x 4096 x 4096: 64 x 64 10.6,
// 128 x 32 12.5; 128 x 4096 x 14336: 128 x 96 22.8, 64 x 192 23.7.
inline Tiling linear_tiling(ProductKind kind, int64_t M, int64_t N, int64_t blocks, int64_t outputs, bool lines) {
    constexpr int64_t kSms = 152;
    const int64_t rate = lines ? 80 : 45;
    const int64_t unit = kind == kGradX || kind == kGradW ? 64 : kind == kGatedFwd ? 32 : 16;
    const int64_t cols = kind == kGatedFwd ? 2 * N : N;
    auto cycles = [&](int64_t tiles, int64_t at_once, int64_t block, int64_t bn) {
        return (tiles + at_once - 1) / at_once * std::max(blocks * block, 12 * bn) + 12 * bn;
    };
    auto single = [&](int64_t high) {
        const int64_t rows = (M + high - 1) / high * outputs, per_row = std::max<int64_t>(1, kSms / rows);
        const int64_t across = per_row * ((cols + 256 * per_row - 1) / (256 * per_row));  // column tiles, of 256 at most
        const int64_t bn = std::min<int64_t>(256, ((cols + across - 1) / across + unit - 1) / unit * unit);
        const int64_t copied = kind == kGradW ? 128 : std::min(high, (M + 7) / 8 * 8), bytes = (copied + bn) * 128;
        const int64_t deep = std::max<int64_t>(1, std::min<int64_t>(kMostDeep, kStageBytes / 4 / bytes));
        const int64_t block = std::max<int64_t>({2 * bn, high + bn, bytes / rate, 140 + 310 / deep});
        return Tiling{1, static_cast<int>(high), static_cast<int>(bn), cycles(rows * ((cols + bn - 1) / bn), kSms, block, bn)};
    };
    if (kind != kGradW && M <= 64) return single(64);
    Tiling best = single(128);
    if (M > 128) {
        const int64_t pair_rows = (M + 255) / 256 * outputs;
        const int64_t narrow_tiles = pair_rows * ((cols + 127) / 128);
        const int64_t narrow_block = narrow_tiles <= kSms / 2 ? (kind == kGradW ? 290 : 270) : (kind == kGradW ? 390 : 340);
        const Tiling narrow{2, 128, 128, cycles(narrow_tiles, kSms / 2, lines ? narrow_block : 540, 128) + 900};
        const Tiling wide{2, 128, 256, cycles(pair_rows * ((cols + 255) / 256), kSms / 2, lines ? 512 : 700, 256) + 900};
        if (narrow.cycles <= best.cycles) best = narrow;
        if (wide.cycles <= best.cycles) best = wide;
    }
    if (kind != kGradW) {
        const Tiling low = single(64);
        if (low.cycles < best.cycles) best = low;
    }
    return best;
}

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
