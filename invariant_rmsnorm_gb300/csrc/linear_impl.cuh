// Matrix products of the projections on the fifth-generation tensor cores: kernel
// and launcher, included by the translation units that instantiate them (linear_fwd,
// linear_grad: bf16; with _f16: fp16).
//
// Mathematics: C = A B^T, its epilogue by kind (linear_launch.h). Every value of C is
// one chain of tensor-core sums over the reduced axis in ascending order, 16 at a
// time, whatever the tile's size, so a row's bits do not depend on M.
//
// A tile of C belongs to a CTA (CTAS = 1: 64 or 128 rows, `bn` columns) or to a pair of CTAs
// (CTAS = 2: 256 rows, 128 or 256 columns; each CTA holds 128 rows of A and half of the columns of B,
// and one instruction multiplies both halves); linear_tiling chooses. Three warps copy blocks of 64
// reduced values of A and B by tensor copies into a ring of stages in shared memory, a
// thread issues their products, which accumulate in tensor memory, and eight warps
// take finished accumulators through the epilogue while the next tile's products run into
// the other half of tensor memory. CTAs are persistent and walk the tiles.
//
// Operands whose rows run along the reduced axis (A, B of the forward, A of kGradX) are
// stages of rows of 128 bytes, the others (B of kGradX, A and B of kGradW) of blocks of 64
// columns: [64 reduced values][128 bytes]. Both are 128-byte swizzled, and zeros are
// filled in beyond the matrix, in both operands alike.
//
// What bounds it. Many rows: the tensor cores, busy 94 to 96 % of a kernel's time (8192 x 4096 x
// 8192: 280 us, 1960 TFLOP/s; back to back for seconds the board's power holds 8192 x 4096 x 16384 at 636 us
// forward, 670 and 666 the gradients, where the library's product takes 622, 655 and 656). Few rows: the issuing
// thread. A product of 16 reduced values reads (rows + columns) x 32 bytes of shared memory, 24 cycles at 64 x 32, 48 at
// 128 x 64; a stage costs the thread 240 more for its wait, descriptors and reconvergence and 75 to 166 for its
// commit. One token of 4096 x 4096: 9.4 us in a graph (5 the reads at the copy rate), 4.3 of them products.
// Between: the operands' way from L2, about 80 bytes a cycle and SM.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "activation.cuh"
#include "kernels.h"
#include "linear_launch.h"

namespace rmsn {
namespace {

constexpr int kBlockK = 64;            // reduced values a block: one swizzled row of 128 bytes
constexpr int kProductThreads = 384;   // warps 0, 2 and 3 copy, 1 multiplies, 2 holds tensor memory, 4 .. 11 epilogue
constexpr int kCopyWarps = 3;          // of a single one's 512 x 4096 x 4096 input gradient 24.9 us, 18.6 of two or three
constexpr int kEpilogueWarps = 8;
constexpr int kMaxStages = 32;
constexpr uint32_t kTileBytes = 32 * 64;             // pairs of CTAs: a warp's piece of the output on its way

// n / d for n < 2^31 by a multiplication (Granlund and Montgomery): a division costs 150 cycles, and a tile's
// first copy waits for three of them.
struct Divisor {
    uint32_t mul, shift;
    __device__ __forceinline__ uint32_t of(uint32_t n) const { return (__umulhi(mul, n) + n) >> shift; }
};
inline Divisor divisor(uint32_t d) {
    uint32_t s = 0;
    while ((uint64_t(1) << s) < d) ++s;
    return {static_cast<uint32_t>((uint64_t(1) << 32) * ((uint64_t(1) << s) - d) / d + 1), s};
}

struct ProductArgs {
    CUtensorMap a[2], b[2];
    CUtensorMap out_map[2], z_map[2];  // pairs of CTAs: boxes of 32 rows of 32 values
    MatOut out[2], z[2];
    MatIn res;
    const float* bias;
    float* partials;
    int64_t M;
    int N;
    int act;
    int tiles_m, tiles_n;     // of one output
    int tiles;                // with the outputs and splits
    Divisor per_output, per_split, per_band, per_last;  // tiles of an output and split, splits, tiles of 8 rows, rows of the last band
    int blocks;               // blocks of the reduced axis
    int segments;             // products that are added (kGradX: 1 or 2)
    int splits;
    int bn;                   // columns of the accumulators of a tile
    int a_rows;               // rows of A in a stage
    int m;                    // rows of the products: 64 or 128 a CTA
    int stages;
    int deep;                 // blocks of 64 reduced values a stage
    int copy_deep;            // blocks a copy (of one matrix): all of a stage's, or one
    bool whole;               // no block is cut short
    uint32_t a_block, b_block, a_bytes, stage_bytes;
    uint32_t idesc;
    int tmem_cols;
    uint32_t staging;         // offset of the epilogue's staging from the ring's start
};

// Device error word of the including translation unit, and whether any of its kernels was launched (or captured): a
// word that nothing can have set is not read, nor its kernels' module loaded for it.
__device__ unsigned int g_linear_error;
std::atomic<bool> g_linear_launched{false};

cudaError_t read_linear_error_word(unsigned* flags, bool clear) {
    if (!g_linear_launched.load()) return cudaSuccess;
    unsigned v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_linear_error, sizeof(v));
    if (e != cudaSuccess) return e;
    *flags |= v;
    if (clear && v) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_linear_error, &zero, sizeof(zero));
    }
    return e;
}

// ---------------------------------------------------------------------------
// Tensor memory and tensor cores
// ---------------------------------------------------------------------------
template <int CTAS>
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {
    if constexpr (CTAS == 2) asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
    else asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
}
template <int CTAS>
__device__ __forceinline__ void tmem_relinquish() {
    if constexpr (CTAS == 2) asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    else asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
template <int CTAS>
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t cols) {
    if constexpr (CTAS == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
    else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
}

// D += A B^T over 16 reduced values (D = A B^T if !add), issued by one thread.
template <int CTAS>
__device__ __forceinline__ void mma16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    if constexpr (CTAS == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add ? 1 : 0) : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add ? 1 : 0) : "memory");
}

// Arrive on `bar` (in both CTAs of a pair) once the thread's earlier products are done.
template <int CTAS>
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    if constexpr (CTAS == 2)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                     ::"r"(smem_u32(bar)), "h"(static_cast<uint16_t>(3)) : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// 16 adjacent columns of this lane's row of the accumulators.
__device__ __forceinline__ void tmem_ld16(uint32_t tmem, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(tmem));
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Shared-memory descriptor: 128-byte swizzle, groups of 8 rows 1024 bytes apart,
// blocks of 64 columns (operands along their columns) `block` bytes apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t at, uint32_t block) {
    return static_cast<uint64_t>((at >> 4) & 0x3fffu) | static_cast<uint64_t>(block >> 4) << 16 |
           static_cast<uint64_t>(1024u >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

// A warp's 32 rows of 32 values from shared memory to the output; beyond the matrix nothing is written.
__device__ __forceinline__ void tile_s2g(const CUtensorMap* map, int c0, int c1, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];"
                 ::"l"(map), "r"(c0), "r"(c1), "r"(src) : "memory");
}
__device__ __forceinline__ void st_shared_v4(uint32_t at, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// A tensor copy into this CTA; a pair's copies count on the first CTA's barrier (`bar`: its
// shared::cluster address).
template <int CTAS>
__device__ __forceinline__ void tile_g2s(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
    if constexpr (CTAS == 2)
        asm volatile(
                        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];"
            ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(bar) : "memory");
    else
        asm volatile(
                        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
            ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(bar) : "memory");
}

// The same of several blocks of 64 columns at once: [blocks][rows][64], for single CTAs.
__device__ __forceinline__ void tile3_g2s(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
                "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar) : "memory");
}
// Arrive on a barrier of the pair's first CTA. Relaxed: it orders no memory but tensor memory, whose reads are
// complete and fenced; a release at cluster scope waits for the output's copies (8192 x 256 x 4096: 30.4 us for 18.7).
__device__ __forceinline__ void cluster_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// True in one lane of a converged warp. (The loops around tensor instructions are
// run by the whole warp, so that their operands stay in uniform registers.)
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p;
}

template <int CTAS>
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity) {
    return mbar_wait_scoped<CTAS == 2>(bar, parity, kWaitTimeoutNs);
}

// ---------------------------------------------------------------------------
// Tiles
// ---------------------------------------------------------------------------
struct Tile { int m, n, which, split; };

// The blocks of the reduced axis that a split has.
__device__ __forceinline__ int2 blocks_of(const ProductArgs& g, int split) {
    if (g.splits == 1) return make_int2(0, g.blocks);
    const uint32_t b = g.blocks;  // at most 2^25 blocks and 64 splits: the product fits 32 bits
    return make_int2(static_cast<int>(g.per_split.of(b * split)), static_cast<int>(g.per_split.of(b * (split + 1))));
}

// Output and split outermost; then bands of 8 rows of tiles, whose operands stay in
// L2 while the band's columns are walked.
__device__ __forceinline__ Tile tile_of(const ProductArgs& g, int t) {
    Tile o{0, 0, 0, 0};
    const uint32_t each = g.tiles_m * g.tiles_n;
    uint32_t u = t;
    if (u >= each) {
        const uint32_t s = g.per_output.of(u);
        u -= s * each;
        o.which = g.per_split.of(s);
        o.split = s - o.which * g.splits;
    }
    const uint32_t b = g.tiles_m > 8 ? g.per_band.of(u) : 0u;
    u -= b * 8 * g.tiles_n;
    const uint32_t rows = min(8u, g.tiles_m - 8 * b);
    o.n = rows == 8 ? u >> 3 : g.per_last.of(u);
    o.m = 8 * b + u - o.n * rows;
    return o;
}

// ---------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------
template <int KIND, int CTAS, bool F16>
__global__ void __launch_bounds__(kProductThreads, 1) product_kernel(const __grid_constant__ ProductArgs g) {
    constexpr bool A_COLS = KIND == kGradW, B_COLS = KIND == kGradX || KIND == kGradW;  // rows across the reduced axis
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drained;
    __shared__ uint32_t tmem_slot;
    // From lane 0, so that what depends on it is known to be the same for the whole warp.
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t rank = CTAS == 2 ? cluster_ctarank() : 0u;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int first_tile = CTAS == 2 ? cluster_id_x() : blockIdx.x, tile_step = CTAS == 2 ? cluster_count_x() : gridDim.x;

    if (warp == 0) {
        if (lane < g.stages) {
            mbar_init(&full[lane], 1);
            mbar_init(&empty[lane], 1);
        }
        if (lane < 2) {
            mbar_init(&acc_full[lane], 1);
            mbar_init(&acc_empty[lane], kEpilogueWarps * CTAS);
        }
        if (lane == 0) mbar_init(&drained, 1);
        fence_mbar_init();
        if (lane < 4) prefetch_tensormap(lane < 2 ? &g.a[lane] : &g.b[lane - 2]);
        __syncwarp();
    } else if (warp == 2) {
        tmem_alloc<CTAS>(smem_u32(&tmem_slot), g.tmem_cols);
        tmem_relinquish<CTAS>();
    }
    tmem_fence_before();
    if constexpr (CTAS == 2) {
        __syncthreads();
        cluster_sync_all();
    } else if (warp == 0) {
        // The first copies need no tensor memory: this warp does not wait for it.
        asm volatile("barrier.cta.arrive 1, %0;" ::"n"(kProductThreads) : "memory");
    } else {
        asm volatile("barrier.cta.sync 1, %0;" ::"n"(kProductThreads) : "memory");
    }
    tmem_fence_after();
    pdl_wait();

    if (warp == 0 || warp == 2 || warp == 3) {
        {  // copies
            // The stages in turn: a copy costs its warp 150 to 200 cycles, as much as a small tile's products of a block.
            const int mine_of = warp == 0 ? 0 : warp - 1;
            int turn = 0;
            int s = 0;
            uint32_t phase = 0;
            int64_t sent = 0;
            bool ok = true;
            const uint32_t all_bytes = g.stage_bytes * CTAS;
            const uint32_t one = elect_one();
            const int deep = g.deep;
            for (int t = first_tile; ok && t < g.tiles; t += tile_step) {
                const Tile c = tile_of(g, t);
                const int2 range = blocks_of(g, c.split);
                const int k0 = range.x, k1 = range.y;
                const int row = c.m * CTAS * g.m + rank * 128;
                for (int seg = 0; ok && seg < g.segments; ++seg) {
                    const CUtensorMap* ma = &g.a[KIND == kGradW ? c.which : seg];
                    for (int k = k0; k < k1; k += deep) {
                        const int now = s;
                        const uint32_t was = phase;
                        const bool skip = turn != mine_of;
                        turn = turn + 1 == kCopyWarps ? 0 : turn + 1;
                        if (++s == g.stages) {
                            s = 0;
                            phase ^= 1u;
                        }
                        ++sent;
                        if (skip) continue;
                        if (!wait_on<CTAS>(&empty[now], was ^ 1u)) {
                            ok = false;
                            break;
                        }
                        if (one) {
                            if (rank == 0) mbar_arrive_expect_tx(&full[now], all_bytes);
                            const uint32_t bar = CTAS == 2 ? cluster_map(&full[now], 0) : smem_u32(&full[now]);
                            const uint32_t at = ring + now * g.stage_bytes, bt = at + g.a_bytes;
                            // Columns of the accumulators: kGatedFwd has half of them of gate, half of up.
                            const int half = g.bn >> 1, mine = g.bn / CTAS, col = c.n * g.bn + rank * mine;
                            // One block (single CTAs: or, along a third axis, all of a stage's) of rows. Blocks past the
                            // last are zeros, or another split's, and not multiplied.
                            auto at_block = [&](int j) { return static_cast<int>(static_cast<uint32_t>(k + j) * kBlockK); };
                            auto rows_of = [&](uint32_t to, const CUtensorMap* map, int r, int j) {
                                if constexpr (CTAS == 2) tile_g2s<CTAS>(to, map, at_block(j), r, bar);
                                else tile3_g2s(to, map, g.whole ? 0 : at_block(j), r, g.whole ? k + j : 0, bar);
                            };
                            auto cols_of = [&](uint32_t to, const CUtensorMap* map, int first, int n, int j) {
                                for (int i = 0; i < n; i += 64) tile_g2s<CTAS>(to + i * 128, map, first + i, at_block(j), bar);
                            };
                            if constexpr (A_COLS) {
                                for (int j = 0; j < deep; ++j) cols_of(at + j * g.a_block, ma, row, 128, j);
                            } else {
                                for (int j = 0; j < deep; j += g.copy_deep) rows_of(at + j * g.a_block, ma, row, j);
                            }
                            if constexpr (B_COLS) {
                                for (int j = 0; j < deep; ++j) cols_of(bt + j * g.b_block, &g.b[seg], col, mine, j);
                            } else if constexpr (KIND == kGatedFwd) {
                                for (int j = 0; j < deep; ++j) {
                                    rows_of(bt + j * g.b_block, &g.b[CTAS == 2 ? rank : 0], c.n * half, j);
                                    if constexpr (CTAS == 1) rows_of(bt + j * g.b_block + half * 128, &g.b[1], c.n * half, j);
                                }
                            } else {
                                for (int j = 0; j < deep; j += g.copy_deep) rows_of(bt + j * g.b_block, &g.b[0], col, j);
                            }
                        }
                        __syncwarp();
                    }
                }
            }
            // Every stage is free again: no arrival on this CTA's barriers is left.
            for (int i = 0; ok && i < g.stages; ++i) {
                ok = wait_on<CTAS>(&empty[s], phase ^ 1u);
                if (++s == g.stages) {
                    s = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) {
                // Give up: wait (bounded) for the copies in flight. A pair's count on its first
                // CTA, so the second waits a millisecond, a thousand times what a copy takes.
                if (one) atomicOr(&g_linear_error, kErrWaitTimeout);
                if (rank == 0) {
                    for (int64_t i = sent > g.stages ? sent - g.stages : 0; i < sent; ++i)
                        (void)wait_on<CTAS>(&full[i % g.stages], static_cast<uint32_t>(i / g.stages) & 1u);
                }
                const unsigned long long t0 = global_timer_ns();
                while (global_timer_ns() - t0 < 1000000ull) {}
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            const uint32_t one = elect_one();
            const int deep = g.deep;
            int s = 0, n = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int t = first_tile; ok && t < g.tiles; t += tile_step, ++n) {
                const int2 range = blocks_of(g, g.splits == 1 ? 0 : tile_of(g, t).split);
                const int blocks = range.y - range.x, buf = n & 1;
                if (!wait_on<CTAS>(&acc_empty[buf], ((n >> 1) & 1) ^ 1u)) {
                    ok = false;
                    break;
                }
                tmem_fence_after();
                const uint32_t d = tmem_slot + buf * g.bn;
                for (int seg = 0; ok && seg < g.segments; ++seg) {
                    for (int k = 0; k < blocks; k += deep) {
                        if (!wait_on<CTAS>(&full[s], phase)) {
                            ok = false;
                            break;
                        }
                        tmem_fence_after();
                        const uint32_t at = ring + s * g.stage_bytes, bt = at + g.a_bytes;
                        const uint64_t da = smem_desc(at, A_COLS ? 8192u : 16u), db = smem_desc(bt, B_COLS ? 8192u : 16u);
                        uint64_t* const used = &empty[s];
                        if (++s == g.stages) {
                            s = 0;
                            phase ^= 1u;
                        }
                        // 16 reduced values: 32 bytes of a row, or two groups of 8 rows.
                        constexpr uint32_t step_a = (A_COLS ? 2048 : 32) >> 4, step_b = (B_COLS ? 2048 : 32) >> 4;
                        if (one) {
#pragma unroll
                            for (int j = 0; j < (CTAS == 2 ? kMostDeepPair : kMostDeep); ++j) {
                                if (j >= min(deep, blocks - k)) break;
#pragma unroll
                                for (int i = 0; i < kBlockK / 16; ++i)
                                    mma16<CTAS>(d, da + j * (g.a_block >> 4) + i * step_a, db + j * (g.b_block >> 4) + i * step_b, g.idesc,
                                                seg > 0 || k > 0 || i > 0 || j > 0);
                            }
                            mma_commit<CTAS>(used);
                        }
                        __syncwarp();
                    }
                }
                if (ok && one) mma_commit<CTAS>(&acc_full[buf]);
                __syncwarp();
            }
            if (!ok) {  // wait (bounded) for the products in flight
                if (one) {
                    atomicOr(&g_linear_error, kErrWaitTimeout);
                    mma_commit<CTAS>(&drained);
                }
                (void)wait_on<CTAS>(&drained, 0);
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        const int quad = warp & 3, part = (warp - 4) >> 2;  // a warp reads the lanes of its quarter
        const uint32_t staged = ring + g.staging + (warp - 4) * 2 * kTileBytes;
        uint32_t piece = 0;
        int n = 0;
        for (int t = first_tile; t < g.tiles; t += tile_step, ++n) {
            const Tile c = tile_of(g, t);
            const int buf = n & 1;
            if (!__all_sync(0xffffffffu, wait_on<CTAS>(&acc_full[buf], (n >> 1) & 1))) {
                if (lane == 0) atomicOr(&g_linear_error, kErrWaitTimeout);
                break;
            }
            tmem_fence_after();
            // Products of 64 rows leave 16 of them in each quarter's first lanes.
            const int lanes = CTAS == 1 && !A_COLS && g.m == 64 ? 16 : 32;
            const int64_t row0 = static_cast<int64_t>(c.m) * CTAS * g.m + rank * 128 + quad * lanes, row = row0 + lane;
            const bool there = lane < lanes && row < g.M;
            const uint32_t acc = tmem_slot + buf * g.bn + (static_cast<uint32_t>(quad * 32) << 16);
            constexpr bool GATED = KIND == kGatedFwd;
            const int width = GATED ? g.bn >> 1 : g.bn;
            if (row0 < g.M) {
                // W columns at a time. Single CTAs write them from the registers, 16 bytes a lane. A pair's, whose
                // output is a large part of the traffic, go through shared memory (rows of 64 bytes, swizzled) and leave
                // by tensor copies, in whole sectors: 8192 x 4096 x 16384 with z kept 591 us from registers, 566 so.
                constexpr int W = CTAS == 2 ? 32 : 16;
                for (int j = part * W; j < width; j += 2 * W) {
                    const int col = c.n * width + j;
                    if (col >= g.N) break;
                    float v[W], u[GATED ? W : 1];
#pragma unroll
                    for (int i = 0; i < W; i += 16) {
                        tmem_ld16(acc + j + i, reinterpret_cast<float(&)[16]>(v[i]));
                        if constexpr (GATED) tmem_ld16(acc + width + j + i, reinterpret_cast<float(&)[16]>(u[i]));
                    }
                    tmem_wait_ld();
                    const int groups = min(W / 8, (g.N - col) >> 3);
                    if constexpr (KIND == kForward) {
                        if (g.bias != nullptr) {
#pragma unroll
                            for (int i = 0; i < W / 4; ++i) {
                                if (i < 2 * groups) {
                                    const float4 b = __ldg(reinterpret_cast<const float4*>(g.bias + col) + i);
                                    v[4 * i] = fadd(v[4 * i], b.x);
                                    v[4 * i + 1] = fadd(v[4 * i + 1], b.y);
                                    v[4 * i + 2] = fadd(v[4 * i + 2], b.z);
                                    v[4 * i + 3] = fadd(v[4 * i + 3], b.w);
                                }
                            }
                        }
                    }
                    auto put = [&](const MatOut& o, const CUtensorMap* map, const float* x) {
                        if constexpr (CTAS == 2) {
                            // The two pieces in turn: the one before the last has been read.
                            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                            __syncwarp();
                            const uint32_t to = staged + piece * kTileBytes;
                            piece ^= 1u;
#pragma unroll
                            for (int i = 0; i < W / 8; ++i)
                                st_shared_v4(to + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4), pack_act<F16>(reinterpret_cast<const float(&)[8]>(x[8 * i])));
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) {
                                tile_s2g(map, col, static_cast<int>(row0), to);
                                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                            }
                        } else if (there) {
                            uint4* p = reinterpret_cast<uint4*>(o.p + row * o.ld + col);
#pragma unroll
                            for (int i = 0; i < W / 8; ++i)
                                if (i < groups) p[i] = pack_act<F16>(reinterpret_cast<const float(&)[8]>(x[8 * i]));
                        }
                    };
                    if constexpr (KIND == kForward || GATED) {
                        if (g.z[0].p != nullptr) put(g.z[0], &g.z_map[0], v);
                        if constexpr (GATED) {
                            if (g.z[1].p != nullptr) put(g.z[1], &g.z_map[1], u);
                        }
                        with_act(g.act, [&](auto act) {
#pragma unroll
                            for (int i = 0; i < W; ++i) v[i] = act_value<decltype(act)::value>(v[i]);
                        });
                        if constexpr (GATED) {
#pragma unroll
                            for (int i = 0; i < W; ++i) v[i] = fmul(v[i], u[i]);
                        }
                        if constexpr (KIND == kForward) {
                            if (g.res.p != nullptr && there) {
                                const uint4* p = reinterpret_cast<const uint4*>(g.res.p + row * g.res.ld + col);
#pragma unroll
                                for (int h = 0; h < W / 8; ++h) {
                                    if (h < groups) {
                                        float r[8];
                                        unpack_act<F16>(p[h], r);
#pragma unroll
                                        for (int i = 0; i < 8; ++i) v[8 * h + i] = fadd(v[8 * h + i], r[i]);
                                    }
                                }
                            }
                        }
                        put(g.out[0], &g.out_map[0], v);
                    } else if (KIND == kGradW && g.splits > 1) {
                        if (there) {
                            float4* p = reinterpret_cast<float4*>(
                                g.partials + ((static_cast<int64_t>(c.which) * g.splits + c.split) * g.M + row) * g.N + col);
#pragma unroll
                            for (int i = 0; i < W / 4; ++i)
                                if (i < 2 * groups) p[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                        }
                    } else {
                        const int which = KIND == kGradW ? c.which : 0;
                        put(g.out[which], &g.out_map[which], v);
                    }
                }
            }
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CTAS == 2) cluster_arrive(cluster_map(&acc_empty[buf], 0));
                else asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&acc_empty[buf])) : "memory");
            }
        }
        if (CTAS == 2 && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }
    pdl_release();
    tmem_fence_before();
    __syncthreads();
    if constexpr (CTAS == 2) cluster_sync_all();
    tmem_fence_after();
    if (warp == 2) tmem_free<CTAS>(tmem_slot, g.tmem_cols);
}

// ---------------------------------------------------------------------------
// Launcher
// ---------------------------------------------------------------------------
template <int KIND, int CTAS, bool F16>
cudaError_t product_run(const Product& p, const Tiling& tile, cudaStream_t st) {
    constexpr bool A_COLS = KIND == kGradW, B_COLS = KIND == kGradX || KIND == kGradW;
    ProductArgs g{};
    const int bn = tile.bn;
    const int width = KIND == kGatedFwd ? bn / 2 : bn;  // columns of C a tile
    g.m = tile.rows;
    const int64_t rows = static_cast<int64_t>(g.m) * CTAS, pairs = KIND == kGradW && p.a[1].p != nullptr ? 2 : 1;
    g.M = p.M;
    g.N = static_cast<int>(p.N);
    g.act = p.act;
    g.splits = p.splits;
    g.segments = KIND == kGradX && p.a[1].p != nullptr ? 2 : 1;
    const int64_t tiles_m = (p.M + rows - 1) / rows, tiles_n = (p.N + width - 1) / width;
    const int64_t tiles = tiles_m * tiles_n * pairs * p.splits, blocks = (p.K + kBlockK - 1) / kBlockK;
    if (tiles >= (int64_t(1) << 30)) return cudaErrorInvalidValue;
    g.tiles_m = static_cast<int>(tiles_m);
    g.tiles_n = static_cast<int>(tiles_n);
    g.tiles = static_cast<int>(tiles);
    g.blocks = static_cast<int>(blocks);
    g.per_output = divisor(static_cast<uint32_t>(tiles_m * tiles_n));
    g.per_split = divisor(static_cast<uint32_t>(p.splits));
    g.per_band = divisor(static_cast<uint32_t>(8 * tiles_n));
    g.per_last = divisor(static_cast<uint32_t>(tiles_m % 8 ? tiles_m % 8 : 8));
    g.bn = bn;
    // Few rows: only those are copied. The products read 64 or 128 rows from the block's start
    // all the same, into what lies behind them in the ring; a row of C depends on its own
    // row of A alone, and the others are not stored. (Products of 64 rows read half of that.)
    const bool few = CTAS == 1 && !A_COLS;
    g.a_rows = few && p.M < g.m ? static_cast<int>((p.M + 7) / 8 * 8) : g.m;
    g.a_block = static_cast<uint32_t>(g.a_rows) * 128u;
    g.b_block = static_cast<uint32_t>(B_COLS ? (bn / CTAS + 63) / 64 * 64 : bn / CTAS) * 128u;
    // Blocks a stage: as many as leave four stages (1 x 4096 x 4096 by 1, 2, 4 and 8 blocks: 18.9, 14.4, 10.5
    // and 9.4 us).
    g.whole = p.K % kBlockK == 0;
    g.deep = std::max(1, std::min<int>(CTAS == 2 ? kMostDeepPair : kMostDeep, static_cast<int>(kStageBytes / 4 / (g.a_block + g.b_block))));
    g.copy_deep = CTAS == 1 && g.whole ? g.deep : 1;
    g.a_bytes = g.a_block * g.deep;
    g.stage_bytes = (g.a_block + g.b_block) * g.deep;
    // What the rows of the last stage's last block reach past the ring.
    const uint32_t reach = (g.deep - 1) * g.a_block + static_cast<uint32_t>(g.m) * 128u;
    const uint32_t behind = std::max(reach, g.stage_bytes) - g.stage_bytes;
    const uint32_t staging = CTAS == 2 ? kEpilogueWarps * 2 * kTileBytes : 0;
    g.stages = std::min<int>(kMaxStages, static_cast<int>((kStageBytes - behind - staging) / g.stage_bytes));
    // A copying warp passes over the others' stages without waiting for them: with fewer stages than such warps
    // it would come to one that is two uses behind, and take its barrier's older phase for the newer.
    if (g.stages < kCopyWarps) return cudaErrorInvalidConfiguration;
    g.staging = static_cast<uint32_t>(g.stages) * g.stage_bytes;
    const size_t smem = static_cast<size_t>(g.staging) + behind + staging + 1024;
    g.tmem_cols = 32;
    while (g.tmem_cols < 2 * bn) g.tmem_cols *= 2;
    // fp32 sums; both operands' format; which of them lie along their columns; N / 8; M / 16.
    g.idesc = 1u << 4 | (F16 ? 0u : 1u) << 7 | (F16 ? 0u : 1u) << 10 | (A_COLS ? 1u : 0u) << 15 | (B_COLS ? 1u : 0u) << 16 |
              static_cast<uint32_t>(bn >> 3) << 17 | static_cast<uint32_t>(g.m * CTAS >> 4) << 24;
    for (int i = 0; i < 2; ++i) {
        g.out[i] = p.out[i];
        g.z[i] = p.z[i];
        const MatIn &a = p.a[i].p != nullptr ? p.a[i] : p.a[0], &b = p.b[i].p != nullptr ? p.b[i] : p.b[0];
        // Operands along their columns and a pair's: in two dimensions; the others in three.
        auto rows_map = [&](CUtensorMap* map, const MatIn& o, int64_t n, int box, int deep) {
            if (CTAS == 2) return encode_blocks_2d(map, o.p, n, p.K, o.ld, box);
            return encode_blocks_3d(map, o.p, n, p.K, o.ld, box, g.whole ? deep : 0);
        };
        cudaError_t e = cudaSuccess;
        if (i == 1 && p.a[1].p == nullptr) g.a[1] = g.a[0];
        else e = A_COLS ? encode_blocks_2d(&g.a[i], a.p, p.K, p.M, a.ld, kBlockK) : rows_map(&g.a[i], a, p.M, g.a_rows, g.deep);
        if (e != cudaSuccess) return e;
        if (i == 1 && p.b[1].p == nullptr) g.b[1] = g.b[0];
        else if (B_COLS) e = encode_blocks_2d(&g.b[i], b.p, p.K, p.N, b.ld, kBlockK);
        else if (KIND == kGatedFwd) e = rows_map(&g.b[i], b, p.N, bn / 2, 1);
        else e = rows_map(&g.b[i], b, p.N, bn / CTAS, g.deep);
        if (e != cudaSuccess) return e;
        if (CTAS == 2) {
            if (p.out[i].p != nullptr && p.splits == 1) e = encode_pieces_2d(&g.out_map[i], p.out[i].p, p.M, p.N, p.out[i].ld);
            if (e == cudaSuccess && p.z[i].p != nullptr) e = encode_pieces_2d(&g.z_map[i], p.z[i].p, p.M, p.N, p.z[i].ld);
            if (e != cudaSuccess) return e;
        }
    }
    g.res = p.res;
    g.bias = p.bias;
    g.partials = p.partials;
    const auto kern = product_kernel<KIND, CTAS, F16>;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    int64_t grid;
    if (CTAS == 2) {
        const int64_t n = pair_clusters(reinterpret_cast<const void*>(kern), kProductThreads, static_cast<int>(smem));
        if (n < 1) return cudaErrorInvalidConfiguration;
        grid = 2 * std::min(tiles, n);
    } else {
        grid = std::min<int64_t>(tiles, sm_count());
    }
    g_linear_launched.store(true);
    return launch_kernel_clustered(kern, static_cast<unsigned>(CTAS), static_cast<unsigned>(grid), kProductThreads, smem, st, g);
}

template <int KIND, bool F16>
cudaError_t product_shape(const Product& p, cudaStream_t st) {
    const int64_t outputs = KIND == kGradW && p.a[1].p != nullptr ? 2 : 1, blocks = (p.K + kBlockK - 1) / kBlockK;
    bool lines = true;  // every row of the operands starts on a line of 128 bytes
    for (const MatIn& m : {p.a[0], p.a[1], p.b[0], p.b[1]}) lines = lines && m.ld % 64 == 0 && reinterpret_cast<uintptr_t>(m.p) % 128 == 0;
    const Tiling t = linear_tiling(static_cast<ProductKind>(KIND), p.M, p.N, (blocks + p.splits - 1) / p.splits, outputs * p.splits, lines);
    return t.ctas == 2 ? product_run<KIND, 2, F16>(p, t, st) : product_run<KIND, 1, F16>(p, t, st);
}

}  // namespace
}  // namespace rmsn
