// Projections and gated feed-forward blocks, forward and backward: the C-ABI entry
// points, the kernels around the matrix products (gradients of the activations, the
// join of split weight gradients), and the workspaces' layout.
#include <algorithm>

#include "activation.cuh"
#include "checks.h"
#include "linear_launch.h"
#include "reduce_columns.h"

namespace rmsn {

namespace {

constexpr int64_t kMaxWidth = int64_t(1) << 20;
constexpr int64_t kMaxStride = int64_t(1) << 38;  // elements: a tensor map's strides are below 2^40 bytes

// ---------------------------------------------------------------------------
// Gradients of the activations: dz = g act'(z), and with a second projection
// dgate = g up act'(gate), dup = g act(gate), in fp32, rounded once: to 16 bits, as the tensor cores' operands. (The products'
// error is 1.4 times that of one rounding so; a high and a low part of each would keep them whole for twice the products.)
//
// Bound by HBM where the activation is cheap: 6 bytes a value (10 with `up`, 2 for the sums alone). A thread takes 8
// adjacent columns of every 8th row of its CTA's range, a CTA 256 columns; the columns' sums (of dz before it
// is rounded) are joined over the CTA's 8 rows of threads in order, one partial row a range.
// 8192 x 14336 gated, silu: 177 us (1.17 GB, 97 % of the copy rate); 8192 x 16384 with the sums' pass 2: none 52 us
// (76 %), silu 105 (75 %), gelu 140 and gelu_tanh 142 (56 %, 66 % of the issue slots).
// ---------------------------------------------------------------------------
constexpr int kSlopeThreads = 256, kSlopeRows = 8, kSlopeCols = 256;

// Ranges of rows: twelve CTAs an SM of a GPU of 152 over all columns, of 32 rows at least. A
// function of T and N alone, so the order of db's sums is too.
int64_t slope_ranges(int64_t T, int64_t N) {
    const int64_t across = (N + kSlopeCols - 1) / kSlopeCols;
    return std::max<int64_t>(1, std::min<int64_t>((1824 + across - 1) / across, (T + 31) / 32));
}

// A saved z, gate or up. The forward went on with the fp32 value; its fp16 copy is infinite beyond 65504, where
// infinity times zero would leave no number. The slopes have their limits at 65504 already, so where only they are
// taken z is held there (VALUE false: in pairs, db of 8192 x 16384 silu 106 us; in fp32 109, without it 104). A value is read as
// fp32's largest: a zero factor leaves zero, and what grows with it is infinite again in fp16. NaN stays. (bf16 has
// fp32's range: an infinite value was so in the forward.)
template <bool F16, bool VALUE>
__device__ __forceinline__ void unpack_saved(uint4 v, float (&f)[8]) {
    if constexpr (F16 && !VALUE) {
        const auto hold = [](uint32_t& w) {
            asm("{\n\t.reg .b32 t;\n\tmin.NaN.f16x2 t, %0, %1;\n\tmax.NaN.f16x2 %0, t, %2;\n\t}" : "+r"(w) : "r"(0x7bff7bffu), "r"(0xfbfffbffu));
        };
        hold(v.x); hold(v.y); hold(v.z); hold(v.w);
    }
    unpack_act<F16>(v, f);
    if constexpr (F16 && VALUE) {
        constexpr float most = 3.4028234663852886e38f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            asm("{\n\t.reg .f32 t;\n\tmin.NaN.f32 t, %0, %1;\n\tmax.NaN.f32 %0, t, %2;\n\t}" : "+f"(f[i]) : "f"(most), "f"(-most));
    }
}

template <int ACT, bool GATED, bool F16>
__device__ __forceinline__ void slope_rows(const Slopes& a, int64_t t0, int64_t t1, int col, float (&sum)[8]) {
    constexpr int BATCH = GATED || ACT != LINEAR_ACT_NONE ? 2 : 4;  // rows whose loads are in flight at once
    constexpr bool HAS_Z = GATED || ACT != LINEAR_ACT_NONE;
    const auto load = [](const MatIn& m, int64_t t, int c) { return __ldcs(reinterpret_cast<const uint4*>(m.p + t * m.ld + c)); };
    for (int64_t t = t0; t < t1; t += BATCH * kSlopeRows) {
        uint4 gv[BATCH], zv[BATCH], uv[BATCH];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int64_t r = t + b * kSlopeRows;
            if (r < t1) {
                gv[b] = load(a.g, r, col);
                if constexpr (HAS_Z) zv[b] = load(a.z, r, col);
                if constexpr (GATED) uv[b] = load(a.up, r, col);
            }
        }
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int64_t r = t + b * kSlopeRows;
            if (r < t1) {
                float g[8], z[8];
                unpack_act<F16>(gv[b], g);
                if constexpr (HAS_Z) unpack_saved<F16, GATED>(zv[b], z);
                if constexpr (GATED) {
                    float u[8], dup[8];
                    unpack_saved<F16, true>(uv[b], u);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 v = act_slope<ACT>(z[i]);
                        dup[i] = fmul(g[i], v.x);
                        g[i] = fmul(fmul(g[i], v.y), u[i]);
                    }
                    *reinterpret_cast<uint4*>(a.out[1].p + r * a.out[1].ld + col) = pack_act<F16>(dup);
                } else if constexpr (HAS_Z) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) g[i] = fmul(g[i], act_slope<ACT>(z[i]).y);
                }
                if constexpr (!GATED) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum[i] = fadd(sum[i], g[i]);
                }
                if (a.out[0].p != nullptr) *reinterpret_cast<uint4*>(a.out[0].p + r * a.out[0].ld + col) = pack_act<F16>(g);
            }
        }
    }
}

template <int ACT, bool GATED, bool F16>
__global__ void __launch_bounds__(kSlopeThreads, GATED ? 3 : 4) slopes_kernel(const Slopes a) {
    __shared__ float part[kSlopeRows][kSlopeCols];
    pdl_wait();
    const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
    const int col = blockIdx.x * kSlopeCols + 8 * lane;
    const int64_t t0 = a.T * blockIdx.y / a.ranges, t1 = a.T * (blockIdx.y + 1) / a.ranges;
    float sum[8] = {};
    if (col < a.N) slope_rows<ACT, GATED, F16>(a, t0 + r, t1, col, sum);
    pdl_release();
    if (a.partials == nullptr) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) part[r][8 * lane + i] = sum[i];
    __syncthreads();
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kSlopeCols + threadIdx.x;
    if (c < a.N) {
        float v = part[0][threadIdx.x];
#pragma unroll
        for (int i = 1; i < kSlopeRows; ++i) v = fadd(v, part[i][threadIdx.x]);
        a.partials[blockIdx.y * a.N + c] = v;
    }
}

template <int ACT>
auto slopes_of(bool gated, bool f16) -> void (*)(Slopes) {
    if (gated) return f16 ? slopes_kernel<ACT, true, true> : slopes_kernel<ACT, true, false>;
    return f16 ? slopes_kernel<ACT, false, true> : slopes_kernel<ACT, false, false>;
}

// ---------------------------------------------------------------------------
// A weight gradient of split rows: the splits' fp32 sums, added in order.
// ---------------------------------------------------------------------------
template <bool F16>
__global__ void __launch_bounds__(256) join_kernel(const float* partials, int splits, const MatOut out, int64_t M, int64_t N) {
    pdl_wait();
    const int64_t groups = N / 8, all = M * groups;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < all; i += gridDim.x * 256ll) {
        float v[8] = {};
        for (int s = 0; s < splits; ++s) {
            const float4* p = reinterpret_cast<const float4*>(partials + s * M * N + i * 8);
            const float4 lo = __ldcs(p), hi = __ldcs(p + 1);
            const float u[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = s == 0 ? u[j] : fadd(v[j], u[j]);
        }
        const int64_t row = i / groups;
        *reinterpret_cast<uint4*>(out.p + row * out.ld + (i - row * groups) * 8) = pack_act<F16>(v);
    }
    pdl_release();
}

// ---------------------------------------------------------------------------
// Argument checks
// ---------------------------------------------------------------------------
int check_sizes(int64_t T, int64_t N, int64_t K, int act) {
    if (T < 0 || T >= (int64_t(1) << 31)) return RMSN_EINVAL;
    if (act < LINEAR_ACT_NONE || act > LINEAR_ACT_RELU) return RMSN_EINVAL;
    if (N < 8 || N > kMaxWidth || N % 8 != 0 || K < 8 || K > kMaxWidth || K % 8 != 0) return RMSN_EUNSUPPORTED;
    return RMSN_OK;
}

int check_mat(const void* p, int64_t ld, int64_t cols) {
    if (ld > kMaxStride) return RMSN_EINVAL;
    return check_act(p, ld, cols);
}

// y may be res, with its stride.
int check_in_place(const void* res, int64_t ldr, const void* y, int64_t ldy, int64_t T) {
    return res == y && T > 1 && ldr != ldy ? RMSN_EINVAL : RMSN_OK;
}

// A workspace of which a call takes `need` bytes (none: it may be anything).
int check_ws(const void* ws, size_t ws_bytes, size_t need) {
    if (need == 0) return RMSN_OK;
    if (ws == nullptr || ws_bytes < need) return RMSN_EWORKSPACE;
    return aligned16(ws) ? RMSN_OK : RMSN_EALIGN;
}

// ---------------------------------------------------------------------------
// Workspaces
// ---------------------------------------------------------------------------
constexpr size_t kAlign = 256;
size_t padded(size_t bytes) { return (bytes + kAlign - 1) / kAlign * kAlign; }

// A weight gradient's cycles by the tiles' model, its rows in s ranges, for which the join costs a launch (5000) and the
// partial sums' way to L2 and back (3000 bytes a cycle). It does not fall with `blocks`, of 64 rows.
int64_t split_cycles(int64_t blocks, int64_t N, int64_t K, int64_t outputs, int64_t s) {
    return linear_tiling(kGradW, N, K, (blocks + s - 1) / s, outputs * s, true).cycles + (s > 1 ? 5000 + 8 * s * outputs * N * K / 3000 : 0);
}

constexpr int kMostSplits = 64;
constexpr int64_t kSplitRows = 512;  // of a range, at least

// Ranges of rows that a weight gradient is split into, where its tiles leave SMs without one:
// the power of two with the fewest cycles. A function of the sizes alone.
int weight_splits(int64_t T, int64_t N, int64_t K, int outputs) {
    const int64_t blocks = (T + 63) / 64;
    int best = 1;
    int64_t least = split_cycles(blocks, N, K, outputs, 1);
    for (int s = 2; s <= kMostSplits && T / s >= kSplitRows; s *= 2) {
        const int64_t cycles = split_cycles(blocks, N, K, outputs, s);
        if (cycles < least) {
            least = cycles;
            best = s;
        }
    }
    return best;
}

// Whether s ranges cost less than any fewer at some count of blocks from lo to hi. Both sides do not fall with
// the blocks, so an interval whose cheapest s is no cheaper than its dearest of the others holds none; the rest is halved. `nodes`
// bounds the intervals looked at (near ties of long axes): past it the answer is yes, which costs bytes alone.
bool splits_pay(int64_t lo, int64_t hi, int64_t N, int64_t K, int64_t outputs, int64_t s, int& nodes) {
    const auto others = [&](int64_t blocks) {
        int64_t least = split_cycles(blocks, N, K, outputs, 1);
        for (int64_t f = 2; f < s; f *= 2) least = std::min(least, split_cycles(blocks, N, K, outputs, f));
        return least;
    };
    if (--nodes < 0) return true;
    const int64_t at_lo = split_cycles(lo, N, K, outputs, s), at_hi = split_cycles(hi, N, K, outputs, s), of_hi = others(hi);
    if (at_lo >= of_hi) return false;
    if (at_hi < of_hi || at_lo < others(lo)) return true;
    if (hi - lo < 2) return false;
    const int64_t mid = lo + (hi - lo) / 2;
    return splits_pay(mid, hi, N, K, outputs, s, nodes) || splits_pay(lo, mid, N, K, outputs, s, nodes);
}

// The most ranges of any T up to T_max: nearly equal costs make them fall and rise with T. (Whole blocks: a T within one
// has its ranges, or fewer.)
int most_splits(int64_t T_max, int64_t N, int64_t K, int outputs) {
    const int at_max = weight_splits(T_max, N, K, outputs);
    for (int64_t s = kMostSplits; s > at_max; s /= 2) {
        const int64_t lo = kSplitRows / 64 * s, hi = T_max / 64;
        int nodes = 2048;
        if (lo <= hi && splits_pay(lo, hi, N, K, outputs, s, nodes)) return static_cast<int>(s);
    }
    return at_max;
}

size_t split_bytes(int splits, int64_t N, int64_t K, int outputs) {
    return splits > 1 ? padded(static_cast<size_t>(splits) * outputs * N * K * 4u) : 0;
}

// linear_bwd's with every output: dz; the partial sums of db; those of dw.
size_t bwd_bytes(int64_t T, int64_t N, int64_t K, int act, int splits) {
    return (act == LINEAR_ACT_NONE ? 0 : padded(static_cast<size_t>(T) * N * 2u)) +
           padded(static_cast<size_t>(slope_ranges(T, N)) * N * 4u) + split_bytes(splits, N, K, 1);
}

// linear_gated_bwd's with every output: dgate and dup; the partial sums of dwg, then dwu.
size_t gated_bwd_bytes(int64_t T, int64_t N, int64_t K, int splits) {
    return 2 * padded(static_cast<size_t>(T) * N * 2u) + split_bytes(splits, N, K, 2);
}

cudaError_t grad(bool f16, ProductKind kind, const Product& p, cudaStream_t s) {
    return f16 ? launch_linear_grad_f16(kind, p, s) : launch_linear_grad(kind, p, s);
}

// dw [N][K] = dz^T x, of one or two dz.
cudaError_t weight_grads(bool f16, const MatIn (&dz)[2], const MatIn& x, const MatOut (&dw)[2], float* partials, int64_t T,
                         int64_t N, int64_t K, cudaStream_t s) {
    const int outputs = dz[1].p != nullptr ? 2 : 1;
    Product p{};
    p.a[0] = dz[0]; p.a[1] = dz[1]; p.b[0] = x; p.out[0] = dw[0]; p.out[1] = dw[1];
    p.M = N; p.N = K; p.K = T; p.partials = partials;
    p.splits = weight_splits(T, N, K, outputs);
    cudaError_t e = grad(f16, kGradW, p, s);
    for (int i = 0; i < outputs && e == cudaSuccess && p.splits > 1; ++i)
        e = launch_linear_join(partials + static_cast<int64_t>(i) * p.splits * N * K, p.splits, dw[i], N, K, f16, s);
    return e;
}

cudaError_t zero_rows(const MatOut& o, int64_t rows, int64_t cols, cudaStream_t s) {
    return cudaMemset2DAsync(o.p, static_cast<size_t>(o.ld) * 2u, 0, static_cast<size_t>(cols) * 2u, static_cast<size_t>(rows), s);
}

}  // namespace

cudaError_t launch_linear_slopes(const Slopes& a, bool f16, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.N + kSlopeCols - 1) / kSlopeCols), static_cast<unsigned>(a.ranges));
    cfg.blockDim = dim3(kSlopeThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = RMSN_PDL;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void (*kern)(Slopes) = nullptr;
    switch (a.act) {
        case LINEAR_ACT_SILU: kern = slopes_of<LINEAR_ACT_SILU>(a.up.p != nullptr, f16); break;
        case LINEAR_ACT_SIGMOID: kern = slopes_of<LINEAR_ACT_SIGMOID>(a.up.p != nullptr, f16); break;
        case LINEAR_ACT_GELU: kern = slopes_of<LINEAR_ACT_GELU>(a.up.p != nullptr, f16); break;
        case LINEAR_ACT_GELU_TANH: kern = slopes_of<LINEAR_ACT_GELU_TANH>(a.up.p != nullptr, f16); break;
        case LINEAR_ACT_RELU: kern = slopes_of<LINEAR_ACT_RELU>(a.up.p != nullptr, f16); break;
        default: kern = slopes_of<LINEAR_ACT_NONE>(a.up.p != nullptr, f16); break;
    }
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_linear_join(const float* partials, int splits, const MatOut& out, int64_t M, int64_t N, bool f16,
                               cudaStream_t s) {
    const int64_t grid = std::min<int64_t>((M * (N / 8) + 255) / 256, static_cast<int64_t>(sm_count()) * 8);
    return launch_kernel(f16 ? join_kernel<true> : join_kernel<false>, static_cast<unsigned>(grid), 256, 0, s, partials, splits,
                         out, M, N);
}

}  // namespace rmsn

using namespace rmsn;

extern "C" {

int linear_fwd(const rmsn_act16* x, int64_t ldx, const rmsn_act16* w, int64_t ldw, const float* b, const rmsn_act16* res,
               int64_t ldr, rmsn_act16* y, int64_t ldy, rmsn_act16* z, int64_t ldz, int64_t T, int64_t N, int64_t K, int act,
               int dtype, rmsn_stream stream) {
    int flags = 0;
    RMSN_TRY(dtype_flags(dtype, &flags));
    RMSN_TRY(check_sizes(T, N, K, act));
    if (T == 0) return RMSN_OK;
    RMSN_TRY(check_mat(x, ldx, K));
    RMSN_TRY(check_mat(w, ldw, K));
    RMSN_TRY(check_mat(y, ldy, N));
    if (b != nullptr) RMSN_TRY(check_vec(b));
    if (z != nullptr) RMSN_TRY(check_mat(z, ldz, N));
    if (res != nullptr) {
        RMSN_TRY(check_mat(res, ldr, N));
        RMSN_TRY(check_in_place(res, ldr, y, ldy, T));
    }
    Product p{};
    p.a[0] = {x, ldx}; p.b[0] = {w, ldw}; p.out[0] = {y, ldy}; p.z[0] = {z, ldz}; p.res = {res, ldr}; p.bias = b;
    p.M = T; p.N = N; p.K = K; p.splits = 1; p.act = act;
    return cuda_status(flags ? launch_linear_fwd_f16(kForward, p, stream) : launch_linear_fwd(kForward, p, stream));
}

size_t linear_bwd_workspace_bytes(int64_t T, int64_t N, int64_t K, int act) {
    if (check_sizes(T, N, K, act) != RMSN_OK || T == 0) return 0;
    return bwd_bytes(T, N, K, act, weight_splits(T, N, K, 1));
}

size_t linear_bwd_workspace_bytes_max(int64_t T_max, int64_t N, int64_t K, int act) {
    if (check_sizes(T_max, N, K, act) != RMSN_OK || T_max == 0) return 0;
    return bwd_bytes(T_max, N, K, act, most_splits(T_max, N, K, 1));
}

int linear_bwd(const rmsn_act16* g, int64_t ldg, const rmsn_act16* x, int64_t ldx, const rmsn_act16* w, int64_t ldw,
               const rmsn_act16* z, int64_t ldz, rmsn_act16* dx, int64_t lddx, rmsn_act16* dw, int64_t lddw, float* db, void* ws,
               size_t ws_bytes, int64_t T, int64_t N, int64_t K, int act, int dtype, rmsn_stream stream) {
    int flags = 0;
    RMSN_TRY(dtype_flags(dtype, &flags));
    RMSN_TRY(check_sizes(T, N, K, act));
    if (dw != nullptr) RMSN_TRY(check_mat(dw, lddw, K));
    if (db != nullptr) RMSN_TRY(check_vec(db));
    if (T == 0) {  // the sums over no rows
        cudaError_t e = dw != nullptr ? zero_rows({dw, lddw}, N, K, stream) : cudaSuccess;
        if (e == cudaSuccess && db != nullptr) e = cudaMemsetAsync(db, 0, static_cast<size_t>(N) * 4u, stream);
        return cuda_status(e);
    }
    RMSN_TRY(check_mat(g, ldg, N));
    if (dx != nullptr) {
        RMSN_TRY(check_mat(dx, lddx, K));
        RMSN_TRY(check_mat(w, ldw, K));
    }
    if (dw != nullptr) RMSN_TRY(check_mat(x, ldx, K));
    if (act != LINEAR_ACT_NONE) RMSN_TRY(check_mat(z, ldz, N));
    // Of the workspace, what the wanted outputs take.
    Slopes a{};
    a.g = {g, ldg}; a.z = {z, ldz}; a.T = T; a.N = N; a.ranges = slope_ranges(T, N); a.act = act;
    const size_t of_dz = act != LINEAR_ACT_NONE && (dx != nullptr || dw != nullptr) ? padded(static_cast<size_t>(T) * N * 2u) : 0;
    const size_t of_db = db != nullptr ? padded(static_cast<size_t>(a.ranges) * N * 4u) : 0;
    const size_t need = of_dz + of_db + (dw != nullptr ? split_bytes(weight_splits(T, N, K, 1), N, K, 1) : 0);
    RMSN_TRY(check_ws(ws, ws_bytes, need));
    const bool f16 = flags != 0;
    unsigned char* at = static_cast<unsigned char*>(ws);
    MatIn dz{g, ldg};
    if (of_dz > 0) {
        a.out[0] = {reinterpret_cast<uint16_t*>(at), N};
        dz = {reinterpret_cast<uint16_t*>(at), N};
    }
    if (db != nullptr) a.partials = reinterpret_cast<float*>(at + of_dz);
    at += of_dz + of_db;
    if (a.out[0].p != nullptr || a.partials != nullptr) RMSN_TRY(cuda_status(launch_linear_slopes(a, f16, stream)));
    if (db != nullptr)
        RMSN_TRY(cuda_status(launch_reduce_columns({a.partials, a.ranges, db}, {nullptr, 0, nullptr}, static_cast<int>(N), stream)));
    if (dx != nullptr) {
        Product p{};
        p.a[0] = dz; p.b[0] = {w, ldw}; p.out[0] = {dx, lddx};
        p.M = T; p.N = K; p.K = N; p.splits = 1;
        RMSN_TRY(cuda_status(grad(f16, kGradX, p, stream)));
    }
    if (dw != nullptr)
        RMSN_TRY(cuda_status(weight_grads(f16, {dz, {}}, {x, ldx}, {{dw, lddw}, {}}, reinterpret_cast<float*>(at), T, N, K, stream)));
    return RMSN_OK;
}

int linear_gated_fwd(const rmsn_act16* x, int64_t ldx, const rmsn_act16* wg, int64_t ldwg, const rmsn_act16* wu, int64_t ldwu,
                     rmsn_act16* h, int64_t ldh, rmsn_act16* gate, int64_t ldgate, rmsn_act16* up, int64_t ldup, int64_t T,
                     int64_t N, int64_t K, int act, int dtype, rmsn_stream stream) {
    int flags = 0;
    RMSN_TRY(dtype_flags(dtype, &flags));
    RMSN_TRY(check_sizes(T, N, K, act));
    if (T == 0) return RMSN_OK;
    RMSN_TRY(check_mat(x, ldx, K));
    RMSN_TRY(check_mat(wg, ldwg, K));
    RMSN_TRY(check_mat(wu, ldwu, K));
    RMSN_TRY(check_mat(h, ldh, N));
    if (gate != nullptr || up != nullptr) {
        RMSN_TRY(check_mat(gate, ldgate, N));
        RMSN_TRY(check_mat(up, ldup, N));
    }
    Product p{};
    p.a[0] = {x, ldx}; p.b[0] = {wg, ldwg}; p.b[1] = {wu, ldwu}; p.out[0] = {h, ldh};
    p.z[0] = {gate, ldgate}; p.z[1] = {up, ldup};
    p.M = T; p.N = N; p.K = K; p.splits = 1; p.act = act;
    return cuda_status(flags ? launch_linear_fwd_f16(kGatedFwd, p, stream) : launch_linear_fwd(kGatedFwd, p, stream));
}

size_t linear_gated_bwd_workspace_bytes(int64_t T, int64_t N, int64_t K) {
    if (check_sizes(T, N, K, LINEAR_ACT_NONE) != RMSN_OK || T == 0) return 0;
    return gated_bwd_bytes(T, N, K, weight_splits(T, N, K, 2));
}

size_t linear_gated_bwd_workspace_bytes_max(int64_t T_max, int64_t N, int64_t K) {
    if (check_sizes(T_max, N, K, LINEAR_ACT_NONE) != RMSN_OK || T_max == 0) return 0;
    return gated_bwd_bytes(T_max, N, K, most_splits(T_max, N, K, 2));
}

int linear_gated_bwd(const rmsn_act16* g, int64_t ldg, const rmsn_act16* x, int64_t ldx, const rmsn_act16* wg, int64_t ldwg,
                     const rmsn_act16* wu, int64_t ldwu, const rmsn_act16* gate, int64_t ldgate, const rmsn_act16* up,
                     int64_t ldup, rmsn_act16* dx, int64_t lddx, rmsn_act16* dwg, int64_t lddwg, rmsn_act16* dwu, int64_t lddwu,
                     void* ws, size_t ws_bytes, int64_t T, int64_t N, int64_t K, int act, int dtype, rmsn_stream stream) {
    int flags = 0;
    RMSN_TRY(dtype_flags(dtype, &flags));
    RMSN_TRY(check_sizes(T, N, K, act));
    const bool weights = dwg != nullptr || dwu != nullptr;
    if (weights) {
        RMSN_TRY(check_mat(dwg, lddwg, K));
        RMSN_TRY(check_mat(dwu, lddwu, K));
    }
    if (T == 0) {  // the sums over no rows
        cudaError_t e = weights ? zero_rows({dwg, lddwg}, N, K, stream) : cudaSuccess;
        if (e == cudaSuccess && weights) e = zero_rows({dwu, lddwu}, N, K, stream);
        return cuda_status(e);
    }
    RMSN_TRY(check_mat(g, ldg, N));
    RMSN_TRY(check_mat(gate, ldgate, N));
    RMSN_TRY(check_mat(up, ldup, N));
    if (dx != nullptr) {
        RMSN_TRY(check_mat(dx, lddx, K));
        RMSN_TRY(check_mat(wg, ldwg, K));
        RMSN_TRY(check_mat(wu, ldwu, K));
    }
    if (weights) RMSN_TRY(check_mat(x, ldx, K));
    if (dx == nullptr && !weights) return RMSN_OK;
    const size_t each = padded(static_cast<size_t>(T) * N * 2u);
    RMSN_TRY(check_ws(ws, ws_bytes, 2 * each + (weights ? split_bytes(weight_splits(T, N, K, 2), N, K, 2) : 0)));
    const bool f16 = flags != 0;
    unsigned char* at = static_cast<unsigned char*>(ws);
    uint16_t *dgate = reinterpret_cast<uint16_t*>(at), *dup = reinterpret_cast<uint16_t*>(at + each);
    Slopes a{};
    a.g = {g, ldg}; a.z = {gate, ldgate}; a.up = {up, ldup}; a.out[0] = {dgate, N}; a.out[1] = {dup, N};
    a.T = T; a.N = N; a.ranges = slope_ranges(T, N); a.act = act;
    RMSN_TRY(cuda_status(launch_linear_slopes(a, f16, stream)));
    if (dx != nullptr) {
        Product p{};
        p.a[0] = {dgate, N}; p.a[1] = {dup, N}; p.b[0] = {wg, ldwg}; p.b[1] = {wu, ldwu}; p.out[0] = {dx, lddx};
        p.M = T; p.N = K; p.K = N; p.splits = 1;
        RMSN_TRY(cuda_status(grad(f16, kGradX, p, stream)));
    }
    if (weights)
        RMSN_TRY(cuda_status(weight_grads(f16, {{dgate, N}, {dup, N}}, {x, ldx}, {{dwg, lddwg}, {dwu, lddwu}},
                                          reinterpret_cast<float*>(at + 2 * each), T, N, K, stream)));
    return RMSN_OK;
}

}  // extern "C"
