// zero_linear.cu -- one linear layer of a training program, forward and backward (zero_linear_*):
//   z = x W + bias, y = act(z) + residual;  dz = dy act'(z), dx = dz W^T, dw = x^T dz, dbias = sum dz
//
// The three products are one kernel, D[M, N] = A[M, K] B[N, K]^T, on the fifth-generation tensor
// cores: TMA tiles in 128-byte swizzled shared memory, tcgen05.mma with fp32 accumulators in
// TMEM, and an epilogue that reads them back while the next tile is multiplied.  Either operand
// may be stored along K or along its own rows (the descriptors' major bit), so no weight and no
// activation is transposed in memory: dw reads x and dz as they are.
//
// Operands whose rows do not start on 16 bytes (the TMA rule) are first copied to rows that do;
// dz is written there by the activation's gradient anyway.
//
// Measured on one GB300 (cuBLAS bf16: 1,947 TFLOP/s in a burst, 1,734 sustained under the power cap):
// 8192 x 11008 x 4096 alone 405 us, 1,824 TFLOP/s; 8192 x 2048 x 8192 with bias and residual 191 us a pass,
// 1,440 (3.4 rounds of tiles: the last is split along the inner dimension); the gradients of 4096 -> 11008
// over 8192 tokens 1,029 to 1,038 us, 1,430 in all, of which 82 are dz; of 1001 -> 1603 over 777 tokens, every row
// off the 16-byte grid, 46.6 us.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "zero_mma.cuh"

namespace zero {

cudaError_t take_norm_error(uint32_t* word, void* stream);    // zero_norm.cu
cudaError_t take_gated_error(uint32_t* word, void* stream);   // zero_gated.cu
cudaError_t take_muon_error(uint32_t* word, void* stream);    // zero_muon.cu

namespace {

// Set by a kernel whose bounded wait ran out (zero_operators_check reads and clears it).
__device__ uint32_t g_linear_error;

enum { kVecOut = 1, kVecPre = 2, kVecRes = 4, kVecBias = 8 };

struct Epilogue {
    uint16_t* out;
    uint16_t* pre;               // z, or NULL
    const uint16_t* bias;        // per column, or NULL
    const uint16_t* residual;    // or NULL
    int64_t ld_out, ld_pre, ld_res;
    int32_t act;
    int32_t vec;                 // which of them allow 16-byte accesses at multiples of 8 columns
};

struct GemmParams {
    CUtensorMap a, b;
    Epilogue epi;
    float* partial;              // [split][tail tile][rows][BN] sums of the tiles that are split
    int32_t M, N, k_blocks;
    int32_t full;                // tiles done whole; the tail after them is split along K
    int32_t splits, k_per_split; // k_blocks of one part (the last may have fewer)
    int32_t tiles_m, tiles_n;
    int32_t a_rows;              // rows of A a copy brings (kBM, or fewer where A has no more)
    int32_t a_mn, b_mn;          // operand stored along its own rows (M or N) instead of along K
    int32_t rows_vec;            // the outputs and the residual allow 16-byte accesses
    uint32_t idesc;
};

// z: the product; bias, activation and residual in fp32, each output rounded once.
template <int DT>
__device__ __forceinline__ void finish8(const Epilogue& E, int64_t row, int64_t col, int n, float (&z)[8],
                                        const float (&bias)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] += bias[j];
    if (E.pre) store8<DT>(E.pre + row * E.ld_pre + col, E.vec & kVecPre, n, z);
    if (E.act != ZERO_ACT_NONE) act_values(z, E.act);
    if (E.residual) {
        float r[8];
        load8<DT>(E.residual + row * E.ld_res + col, E.vec & kVecRes, n, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] += r[j];
    }
    store8<DT>(E.out + row * E.ld_out + col, E.vec & kVecOut, n, z);
}

// One element.
template <int DT>
__device__ __forceinline__ void finish1(const Epilogue& E, int64_t row, int64_t col, float z)
{
    if (E.bias) z += widen1<DT>(E.bias[col]);
    if (E.pre) E.pre[row * E.ld_pre + col] = narrow1<DT>(z);
    z = act_value(z, E.act);
    if (E.residual) z += widen1<DT>(E.residual[row * E.ld_res + col]);
    E.out[row * E.ld_out + col] = narrow1<DT>(z);
}

template <int DT>
__device__ __forceinline__ void bias8(const Epilogue& E, int64_t col, int n, float (&b)[8])
{
    if (E.bias && n > 0) {
        load8<DT>(E.bias + col, E.vec & kVecBias, n, b);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = 0.0f;
    }
}

// ------------------------------------------------------------------ the product

// Work item `item`: a tile and its inner blocks [kb0, kb1); part >= 0: its place among the partial sums.
struct Item {
    int m, n, kb0, kb1, part;
};

__device__ __forceinline__ Item item_at(const GemmParams& P, int item)
{
    Item I;
    const int tail = P.tiles_m * P.tiles_n - P.full;
    int tile = item, split = 0;
    I.part = -1;
    if (item >= P.full && P.splits > 1) {
        I.part = item - P.full;
        split = I.part / tail;
        tile = P.full + I.part - split * tail;
    }
    tile_at(P.tiles_m, P.tiles_n, tile, I.m, I.n);
    I.kb0 = I.part >= 0 ? split * P.k_per_split : 0;
    I.kb1 = I.part >= 0 ? min(P.k_blocks, I.kb0 + P.k_per_split) : P.k_blocks;
    return I;
}

// CG = 2: the two blocks of a cluster form one 256 x BN tile: each stages 128 rows of A and BN / 2
// of B, the first one issues products that read both, and each keeps the accumulators of its own
// 128 rows.  CG = 1: one block, 128 x BN.
template <int CG, int BN, int DT>
__global__ void __cluster_dims__(CG, 1, 1) __launch_bounds__(kGemmThreads, 1)
    gemm_kernel(const __grid_constant__ GemmParams P)
{
    using S = GemmShape<CG, BN>;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = (uint32_t)__cvta_generic_to_shared(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t epi0 = base + S::kStages * S::kStageBytes;
    const uint32_t bars = epi0 + kEpiWarps * kEpiBytes;
    const uint32_t full0 = bars, empty0 = full0 + 8 * S::kStages, acc_full0 = empty0 + 8 * S::kStages,
                   acc_empty0 = acc_full0 + 16, tmem_slot = acc_empty0 + 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0;
    const int n_items = P.full + (P.tiles_m * P.tiles_n - P.full) * P.splits;
    const int first = blockIdx.x / CG, step = gridDim.x / CG;

    if (warp == 0 && lane == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full0 + 8 * i, 1);
            mbar_init(acc_empty0 + 8 * i, kEpiWarps * CG);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&P.a) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&P.b) : "memory");
    }
    if (warp == 2) {
        if constexpr (CG == 2) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tmem_slot), "n"(S::kTmemCols) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tmem_slot), "n"(S::kTmemCols) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tmem_slot));
    after_earlier_work();

    bool ok = true;
    if (warp == 0) {
        // ---- producer: one thread
        if (lane == 0) {
            uint32_t k = 0;
            for (int item = first; item < n_items && ok; item += step) {
                const Item I = item_at(P, item);
                const int row_a = (I.m * CG + (int)rank) * kBM, row_b = I.n * BN + (int)rank * S::kBRows;
                for (int kb = I.kb0; kb < I.kb1; ++kb, ++k) {
                    const uint32_t s = k % S::kStages, use = k / S::kStages;
                    if (use > 0 && !mbar_wait(empty0 + 8 * s, (use - 1) & 1, kGemmWaitNs)) {
                        ok = false;
                        break;
                    }
                    const uint32_t a = base + s * S::kStageBytes, b = a + S::kABytes;
                    uint32_t bar = full0 + 8 * s;
                    if (rank == 0) mbar_arrive_expect_tx(bar, CG * (P.a_rows * (kBK * 2) + S::kBBytes));
                    if constexpr (CG == 2) bar = leader_address(bar);
                    if (P.a_mn) {
                        for (int i = 0; i < kBM / 64; ++i)
                            tma_load_2d<CG>(a + i * (kBK * 128), &P.a, row_a + 64 * i, kb * kBK, bar);
                    } else {
                        tma_load_2d<CG>(a, &P.a, kb * kBK, row_a, bar);
                    }
                    if (P.b_mn) {
                        for (int i = 0; i < S::kBRows / 64; ++i)
                            tma_load_2d<CG>(b + i * (kBK * 128), &P.b, row_b + 64 * i, kb * kBK, bar);
                    } else {
                        tma_load_2d<CG>(b, &P.b, kb * kBK, row_b, bar);
                    }
                }
            }
        }
    } else if (warp == 1) {
        // ---- products: one thread of the leading block
        if (lane == 0 && rank == 0) {
            uint32_t k = 0, tile = 0;
            for (int item = first; item < n_items && ok; item += step, ++tile) {
                const Item I = item_at(P, item);
                const int kb0 = I.kb0, kb1 = I.kb1;
                const uint32_t acc = tile & 1, use = tile >> 1;
                if (use > 0 && !mbar_wait(acc_empty0 + 8 * acc, (use - 1) & 1, kGemmWaitNs)) {
                    ok = false;
                    break;
                }
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                for (int kb = kb0; kb < kb1; ++kb, ++k) {
                    const uint32_t s = k % S::kStages;
                    if (!mbar_wait(full0 + 8 * s, (k / S::kStages) & 1, kGemmWaitNs)) {
                        ok = false;
                        break;
                    }
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint32_t a = base + s * S::kStageBytes, b = a + S::kABytes;
                    const uint64_t da = smem_desc(a, P.a_mn), db = smem_desc(b, P.b_mn);
                    // 16 inner elements: 32 bytes along K, two groups of eight K rows along MN
                    const uint64_t sa = P.a_mn ? 2048 >> 4 : 32 >> 4, sb = P.b_mn ? 2048 >> 4 : 32 >> 4;
#pragma unroll
                    for (int i = 0; i < kBK / 16; ++i)
                        mma_f16<CG>(tmem + acc * BN, da + sa * i, db + sb * i, P.idesc, kb > kb0 || i > 0);
                    mma_commit<CG>(empty0 + 8 * s);
                }
                if (!ok) break;
                mma_commit<CG>(acc_full0 + 8 * acc);
            }
        }
    } else if (warp >= 4) {
        // ---- epilogue: warp w reads TMEM lanes 32 (w % 4) on; the two warps of a lane group take
        // alternate column chunks
        const int quad = warp & 3, half = (warp - 4) >> 2;
        const uint32_t stage = epi0 + (warp - 4) * kEpiBytes;
        const uint32_t acc_empty_leader = CG == 2 ? leader_address(acc_empty0) : acc_empty0;
        uint32_t tile = 0;
        for (int item = first; item < n_items && ok; item += step, ++tile) {
            const Item I = item_at(P, item);
            const uint32_t acc = tile & 1, use = tile >> 1;
            const int row_in = (int)rank * kBM + quad * 32;                     // of the tile
            const int64_t row0 = (int64_t)I.m * (CG * kBM) + row_in;
            ok = mbar_wait(acc_full0 + 8 * acc, use & 1, kGemmWaitNs);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            for (int c = half * kEpiCols; c < BN; c += 2 * kEpiCols) {
                const int64_t col0 = (int64_t)I.n * BN + c, col = col0 + (lane & 3) * 8;   // this lane's eight columns
                if (col0 >= P.N || row0 >= P.M) break;
                float x[32];
                tmem_load32(tmem + acc * BN + c + ((uint32_t)(quad * 32) << 16), x);
                // transposed through shared memory: 16-byte pieces, exchanged within eight rows so
                // that neither side has bank conflicts
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t at = stage + lane * 128 + ((i ^ (lane & 7)) << 4);
                    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(x[4 * i]), "f"(x[4 * i + 1]),
                                 "f"(x[4 * i + 2]), "f"(x[4 * i + 3])
                                 : "memory");
                }
                __syncwarp();
                if (I.part < 0 && !P.rows_vec) {
                    // rows that do not start on 16 bytes: a column a lane, so that a warp writes neighbours;
                    // eight rows at a time, as a store may not pass an earlier load of the residual
                    if (col0 + lane < P.N) {
                        const int rows = (int)min((int64_t)32, P.M - row0);
                        const Epilogue& E = P.epi;
                        const float bias = E.bias ? widen1<DT>(E.bias[col0 + lane]) : 0.0f;
                        for (int r0 = 0; r0 < rows; r0 += 8) {
                            float z[8], res[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                res[j] = E.residual && r0 + j < rows ? widen1<DT>(E.residual[(row0 + r0 + j) * E.ld_res + col0 + lane]) : 0.0f;
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const uint32_t at = stage + (r0 + j) * 128 + (((lane >> 2) ^ j) << 4) + (lane & 3) * 4;
                                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(z[j]) : "r"(at) : "memory");
                            }
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                if (r0 + j >= rows) break;
                                const int64_t row = row0 + r0 + j;
                                z[j] += bias;
                                if (E.pre) E.pre[row * E.ld_pre + col0 + lane] = narrow1<DT>(z[j]);
                                E.out[row * E.ld_out + col0 + lane] = narrow1<DT>(act_value(z[j], E.act) + res[j]);
                            }
                        }
                    }
                    __syncwarp();
                    continue;
                }
                const int cols = (int)max((int64_t)0, min((int64_t)8, P.N - col));
                float bias[8];
                if (I.part < 0) bias8<DT>(P.epi, col, cols, bias);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = i * 8 + (lane >> 2), p = (lane & 3) * 2;
                    float z[8];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t at = stage + r * 128 + (((p + j) ^ (r & 7)) << 4);
                        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(z[4 * j]), "=f"(z[4 * j + 1]), "=f"(z[4 * j + 2]), "=f"(z[4 * j + 3])
                                     : "r"(at)
                                     : "memory");
                    }
                    const int64_t row = row0 + r;
                    if (row < P.M && cols > 0) {
                        if (I.part >= 0) {
                            float4* q = reinterpret_cast<float4*>(P.partial + ((int64_t)I.part * (CG * kBM) + row_in + r) * BN + c + (lane & 3) * 8);
                            q[0] = make_float4(z[0], z[1], z[2], z[3]);
                            q[1] = make_float4(z[4], z[5], z[6], z[7]);
                        } else {
                            finish8<DT>(P.epi, row, col, cols, z, bias);
                        }
                    }
                }
                __syncwarp();
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                if constexpr (CG == 2) arrive_cluster(acc_empty_leader + 8 * acc);
                else mbar_arrive(acc_empty0 + 8 * acc);
            }
        }
    }
    if (!ok) {
        // A wait ran out: say so, and give copies and products in flight time to end before the
        // block's memory is given back.
        if (lane == 0) atomicOr(&g_linear_error, 1u);
        const uint64_t t0 = global_ns();
        for (uint32_t i = 0; i < kWaitIterCap && global_ns() - t0 < 100000000ull; ++i) __nanosleep(1000);
    }
    __syncwarp();
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (warp == 2) {
        if constexpr (CG == 2)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(S::kTmemCols));
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(S::kTmemCols));
    }
}

// The partial sums of the split tiles, in order, with the epilogue.  A block takes 8 rows of a tile, a
// warp one: eight neighbouring columns a lane, or (rows that do not start on 16 bytes) every 32nd.
struct TailParams {
    const float* partial;
    Epilogue epi;
    int32_t M, N, full, splits, tiles_m, tiles_n, tile_rows, bn, rows_vec;
};

template <int DT>
__global__ void __launch_bounds__(256) tail_sum_kernel(const __grid_constant__ TailParams P)
{
    after_earlier_work();
    const int lane = threadIdx.x & 31, in = blockIdx.x * 8 + (threadIdx.x >> 5);    // the row in its tile
    const int tail = gridDim.y, r = blockIdx.y;
    int m, n;
    tile_at(P.tiles_m, P.tiles_n, P.full + r, m, n);
    const int64_t row = (int64_t)m * P.tile_rows + in, col0 = (int64_t)n * P.bn;
    if (row >= P.M) return;
    const float* from = P.partial + ((int64_t)r * P.tile_rows + in) * P.bn;
    const int64_t next = (int64_t)tail * P.tile_rows * P.bn;
    if (P.rows_vec) {
        const int c = lane * 8, cols = (int)min((int64_t)8, P.N - col0 - c);
        if (c >= P.bn || cols <= 0) return;
        float z[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f}, bias[8];
#pragma unroll 8
        for (int s = 0; s < P.splits; ++s) {
            const float4* q = reinterpret_cast<const float4*>(from + s * next + c);
            const float4 a = __ldcs(q), b = __ldcs(q + 1);
            z[0] += a.x; z[1] += a.y; z[2] += a.z; z[3] += a.w;
            z[4] += b.x; z[5] += b.y; z[6] += b.z; z[7] += b.w;
        }
        bias8<DT>(P.epi, col0 + c, cols, bias);
        finish8<DT>(P.epi, row, col0 + c, cols, z, bias);
    } else {
        for (int c = lane; c < P.bn && col0 + c < P.N; c += 32) {
            float z = 0.0f;
#pragma unroll 4
            for (int s = 0; s < P.splits; ++s) z += __ldcs(from + s * next + c);
            finish1<DT>(P.epi, row, col0 + c, z);
        }
    }
}

// The product over an empty inner dimension: z = 0.
template <int DT>
__global__ void __launch_bounds__(256) empty_sum_kernel(int64_t M, int64_t N, const __grid_constant__ Epilogue E)
{
    after_earlier_work();
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < M * N; i += (int64_t)gridDim.x * 256)
        finish1<DT>(E, i / N, i % N, 0.0f);
}

// ------------------------------------------------------------------ dz, and aligned copies

// What precedes the products, one launch: dz, and the copies of x and of w.
struct DzParams {
    AlignJob copy[2];
    int32_t dz_blocks, across;   // blocks of the dz pass, and how many of them share rows
    int32_t copy_blocks[2];
    const uint16_t* dy;
    const uint16_t* pre;     // NULL: the activation is none
    uint16_t* dz;            // rows of ld_dz elements, 16-byte aligned; NULL: only the sums
    float* sums;             // [worker][ld_dz] column sums, or NULL
    int64_t rows, cols, ld_dy, ld_pre, ld_dz;
    int32_t act, vec_dy, vec_pre, chunk;   // chunk: consecutive rows a worker takes
};

// FLIGHT rows of a thread's eight columns; FULL: all eight are there, by 16-byte accesses.
template <int DT, bool FULL, int FLIGHT>
__device__ __forceinline__ void dz_rows(const DzParams& P, int64_t col, int n, int64_t r, float (&sum)[8])
{
    uint4 d[FLIGHT], z[FLIGHT];
#pragma unroll
    for (int i = 0; i < FLIGHT; ++i) {
        const int64_t row = r + i;
        if constexpr (FULL) {
            d[i] = __ldcs(reinterpret_cast<const uint4*>(P.dy + row * P.ld_dy + col));
            if (P.pre) z[i] = __ldcs(reinterpret_cast<const uint4*>(P.pre + row * P.ld_pre + col));
        } else {
            auto gather = [&](const uint16_t* p) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = (2 * j < n ? p[2 * j] : 0u) | ((2 * j + 1 < n ? (uint32_t)p[2 * j + 1] : 0u) << 16);
                return make_uint4(w[0], w[1], w[2], w[3]);
            };
            d[i] = gather(P.dy + row * P.ld_dy + col);
            if (P.pre) z[i] = gather(P.pre + row * P.ld_pre + col);
        }
    }
#pragma unroll
    for (int i = 0; i < FLIGHT; ++i) {
        float x[8];
        widen2<DT>(d[i].x, x[0], x[1]);
        widen2<DT>(d[i].y, x[2], x[3]);
        widen2<DT>(d[i].z, x[4], x[5]);
        widen2<DT>(d[i].w, x[6], x[7]);
        if (P.pre) {
            float y[8];
            widen2<DT>(z[i].x, y[0], y[1]);
            widen2<DT>(z[i].y, y[2], y[3]);
            widen2<DT>(z[i].z, y[4], y[5]);
            widen2<DT>(z[i].w, y[6], y[7]);
            act_slopes(y, P.act);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= y[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += FULL || j < n ? x[j] : 0.0f;
        if (P.dz) store8<DT>(P.dz + (r + i) * P.ld_dz + col, true, n, x);
    }
}

// dz = dy act'(pre), and its column sums: a thread takes eight columns of a worker's rows (blocks of up to
// 2048 columns; narrower ones hold several workers), so that the sums need no exchange.
template <int DT>
__global__ void __launch_bounds__(256, 4) dz_kernel(const __grid_constant__ DzParams P)
{
    after_earlier_work();
    constexpr int kFlight = 2;
    if ((int)blockIdx.x >= P.dz_blocks) {
        const int b = blockIdx.x - P.dz_blocks;
        const int which = b >= P.copy_blocks[0];
        align_rows(P.copy[which], which ? b - P.copy_blocks[0] : b, P.copy_blocks[which]);
        return;
    }
    const int by = blockIdx.x / P.across, bx = blockIdx.x - by * P.across;
    const int64_t col = ((int64_t)bx * blockDim.x + threadIdx.x) * 8;
    const int n = (int)max((int64_t)0, min((int64_t)8, P.cols - col));
    const int64_t worker = (int64_t)by * blockDim.y + threadIdx.y;
    const int64_t r1 = min(P.rows, (worker + 1) * P.chunk);
    int64_t r = worker * P.chunk;
    if (n == 0 || r >= r1) return;
    float sum[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (n == 8 && P.vec_dy && (P.vec_pre || !P.pre)) {
        for (; r + kFlight <= r1; r += kFlight) dz_rows<DT, true, kFlight>(P, col, n, r, sum);
        for (; r < r1; ++r) dz_rows<DT, true, 1>(P, col, n, r, sum);
    } else {
        for (; r + kFlight <= r1; r += kFlight) dz_rows<DT, false, kFlight>(P, col, n, r, sum);
        for (; r < r1; ++r) dz_rows<DT, false, 1>(P, col, n, r, sum);
    }
    if (!P.sums) return;
    float4* q = reinterpret_cast<float4*>(P.sums + worker * P.ld_dz + col);      // rows of a multiple of 8
    q[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
    q[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
}

// Sums over the workers, in a fixed order, in fp32: 32 columns by 8 workers at a time.
template <int DT>
__global__ void __launch_bounds__(256) column_sum_kernel(const float* sums, int64_t ld, int64_t workers, int64_t cols,
                                                         uint16_t* out, int accumulate)
{
    after_earlier_work();
    __shared__ float part[8][33];
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int64_t w = threadIdx.y; w < workers; w += 8) s += sums[w * ld + c];
    }
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y != 0 || c >= cols) return;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += part[i][threadIdx.x];
    if (accumulate) s += widen1<DT>(out[c]);
    out[c] = narrow1<DT>(s);
}

// ------------------------------------------------------------------ few rows
//
// Up to kFewRows rows of x: reading W is all there is.  fp32 products on the plain cores straight from the
// loads, no tiles and one launch, for operands on the 16-byte grid.  What it costs is not the arithmetic but
// what stands between the loads: none is behind a branch, sums are joined once a warp, and blocks are as many
// as run at one time.  Measured on one GB300 in a graph of such calls, W from HBM, one and two rows (tiles
// need 12.8 us for the first two, 23.6 and 40 for the others):
//   2048 -> 8192   (out, in) 7.3 and 7.7 us, (in, out) 8.2 and 9.4     (33.5 MB: 4.9 at the copy rate)
//   8192 -> 2048             7.3 and 7.7               8.6 and 9.8
//   4096 -> 11008            18.9 and 20.2            16.3 and 18.0
//   2048 -> 50304            35.0 and 36.7            33.3 and 35.7
// Four rows take 14 and 27 us for the first of them: the tiles' from three on.
// (out, in): two loads of two rows a lane and four blocks an SM; four loads and three blocks 8.0 and 9.8 us,
// eight loads of one row 9.2.  (in, out): 256 threads and two parts of K 8.2, four parts (more blocks than
// run at one time) 10.4, blocks of 512 threads 10.3.
constexpr int kFewRows = 2;
constexpr int kFewWarps = 8, kFewCols = 2;            // (out, in): warps a block, rows of W a warp
constexpr int kFewDeep = 8, kFewParts = 8;           // (in, out): warps a block, blocks a cluster at most
constexpr int kFewResident = 3;                       // (in, out): blocks an SM

struct FewParams {
    const uint16_t *x, *w;
    Epilogue epi;
    int64_t ld_x, ld_w;
    int32_t M, N, K;   // K (and N where W is stored along it) in eights; rows of x and W start on 16 bytes
    int32_t split;     // (out, in): warps along K
};

// W stored (out, in): a warp takes kFewCols rows of W and every `split`-th 256 elements of them.
template <int DT, int ROWS>
__global__ void __launch_bounds__(32 * kFewWarps, 4) few_rows_kernel(const __grid_constant__ FewParams P)
{
    constexpr int C = kFewCols, U = 2;
    __shared__ float part[kFewWarps][ROWS * C];
    after_earlier_work();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, ways = P.split, sub = warp % ways;
    const int64_t n0 = ((int64_t)blockIdx.x * (kFewWarps / ways) + warp / ways) * C;
    const uint16_t *x[ROWS], *w[C];   // the last row again where there are fewer
#pragma unroll
    for (int m = 0; m < ROWS; ++m) x[m] = P.x + min(m, P.M - 1) * P.ld_x;
#pragma unroll
    for (int c = 0; c < C; ++c) w[c] = P.w + min(n0 + c, (int64_t)P.N - 1) * P.ld_w;
    F2 acc[ROWS][C];
#pragma unroll
    for (int m = 0; m < ROWS; ++m)
#pragma unroll
        for (int c = 0; c < C; ++c) acc[m][c] = both(0.0f);
    const int64_t step = ways * 256;
    int64_t k = sub * 256 + lane * 8;
    for (; k + (U - 1) * step < P.K; k += U * step) few_eights<DT, U, ROWS, C>(x, w, k, step, acc);
    for (; k < P.K; k += step) few_eights<DT, 1, ROWS, C>(x, w, k, step, acc);
#pragma unroll
    for (int m = 0; m < ROWS; ++m)
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float a, b;
            split(acc[m][c], a, b);
            a += b;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
            if (lane == 0) part[warp][m * C + c] = a;
        }
    __syncthreads();
    const int i = threadIdx.x;
    if (i >= kFewWarps / ways * ROWS * C) return;
    const int g = i / (ROWS * C), m = i % (ROWS * C) / C, c = i % C;
    const int64_t n = ((int64_t)blockIdx.x * (kFewWarps / ways) + g) * C + c;
    if (m >= P.M || n >= P.N) return;
    float z = 0.0f;
    for (int v = 0; v < ways; ++v) z += part[g * ways + v][m * C + c];
    finish1<DT>(P.epi, m, n, z);
}

// W stored (in, out): a block takes 64 columns and one part of K, a thread eight columns and eight rows of W
// at a time, so that its eight elements of x are one load; the blocks of a cluster are the parts, summed in
// order.
template <int DT, int ROWS>
__global__ void __launch_bounds__(32 * kFewDeep, kFewResident) few_rows_deep_kernel(const __grid_constant__ FewParams P)
{
    __shared__ float part[kFewDeep][ROWS * 64];
    __shared__ float whole[ROWS * 64];
    after_earlier_work();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, across = (lane & 7) * 8;
    // past the last column: that column's eight again
    const uint16_t* w = P.w + min((int64_t)blockIdx.x * 64 + across, (int64_t)P.N - 8);
    const int64_t per = (P.K / 8 + gridDim.y - 1) / gridDim.y * 8, end = min((int64_t)P.K, (blockIdx.y + 1) * per);
    F2 acc[ROWS][4];
#pragma unroll
    for (int m = 0; m < ROWS; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[m][j] = both(0.0f);
    for (int64_t k = blockIdx.y * per + warp * 32 + (lane >> 3) * 8; k < end; k += kFewDeep * 32) {
        uint4 wv[8], xv[ROWS];
#pragma unroll
        for (int u = 0; u < 8; ++u) wv[u] = __ldcs(reinterpret_cast<const uint4*>(w + (k + u) * P.ld_w));
#pragma unroll
        for (int m = 0; m < ROWS; ++m) xv[m] = *reinterpret_cast<const uint4*>(P.x + min(m, P.M - 1) * P.ld_x + k);
#pragma unroll
        for (int u = 0; u < 8; u += 2) {
            F2 f[2][4];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float a, b;
                widen2<DT>(word(wv[u + j / 4], j % 4), a, b);
                f[j / 4][j % 4] = pair(a, b);
            }
#pragma unroll
            for (int m = 0; m < ROWS; ++m) {
                float a, b;
                widen2<DT>(word(xv[m], u / 2), a, b);
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[m][j] = fma(both(a), f[0][j], acc[m][j]);
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[m][j] = fma(both(b), f[1][j], acc[m][j]);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < ROWS; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float a, b;
            split(acc[m][j], a, b);
#pragma unroll
            for (int o = 8; o < 32; o *= 2) {
                a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
                b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
            }
            if (lane < 8) {
                part[warp][m * 64 + across + 2 * j] = a;
                part[warp][m * 64 + across + 2 * j + 1] = b;
            }
        }
    __syncthreads();
    const int i = threadIdx.x, m = i / 64;
    const int64_t col = (int64_t)blockIdx.x * 64 + i % 64;
    const bool mine = i < ROWS * 64 && m < P.M && col < P.N;
    float z = 0.0f;
    if (mine) {
#pragma unroll
        for (int v = 0; v < kFewDeep; ++v) z += part[v][i];
    }
    if (gridDim.y > 1) {
        if (mine) whole[i] = z;
        cluster_sync();
        if (mine && blockIdx.y == 0) {
            for (uint32_t r = 1; r < gridDim.y; ++r) {
                uint32_t at;
                float v;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(&whole[i])), "r"(r));
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
                z += v;
            }
        }
        cluster_sync();   // a block's shared memory outlives the reads of it
    }
    if (mine && blockIdx.y == 0) finish1<DT>(P.epi, m, col, z);
}

// ------------------------------------------------------------------ host: one product

// How a product is cut: the tile's shape; tiles done whole, a multiple of what runs at one time; and the
// parts along K that the rest is split into.
struct Cut {
    int cg = 2, bn = 256;
    int splits = 1, per_split = 0;
    int64_t tiles_m = 0, tiles_n = 0, full = 0;
    int64_t tail() const { return tiles_m * tiles_n - full; }
    int64_t tile_elems() const { return (int64_t)kBM * cg * bn; }
};

// The cut with the least estimated time.  One inner block (kBK) of a 256 x 256 tile on a pair of SMs takes
// 0.336 us, 94 % of the tensor cores' measured rate.  A 128 x 128 tile on one SM takes 0.29: the same
// bytes for a quarter of the products (an SM takes 117 GB/s from L2, 64 bytes a clock).  It serves
// where there are few rows or few tiles.  Split tiles write and read fp32 partial sums once (L2), in a
// launch of their own, 2.5 us as it is set up beside the product's (1024 rows, 4096 -> 1024: split 17.3 us,
// whole 21.9; 512 rows, 2048 -> 2048 stay whole, 12.9).
Cut choose_cut(int64_t M, int64_t N, int64_t K)
{
    const int64_t kb = div_up(std::max<int64_t>(K, 1), kBK);
    Cut best;
    double best_us = 1e30;
    static const struct {
        int cg, bn;
        double block_us;
    } shapes[] = {{2, 256, 0.336}, {1, 128, 0.29}, {1, 64, 0.20}};
    for (const auto& shape : shapes) {
        const int cg = shape.cg;
        const double block_us = shape.block_us;
        Cut c;
        c.cg = cg;
        c.bn = shape.bn;
        c.tiles_m = div_up(M, kBM * cg);
        c.tiles_n = div_up(N, c.bn);
        const int64_t slots = kGb300Sms / cg, tiles = c.tiles_m * c.tiles_n;
        for (int64_t want = 1; want <= std::min<int64_t>(kb, 76); ++want) {
            const int64_t per = div_up(kb, want), splits = div_up(kb, per);
            if (splits != want) continue;
            c.full = splits == 1 ? tiles : tiles / slots * slots;
            if (splits > 1 && c.tail() == 0) continue;
            if (splits * c.tail() * c.tile_elems() > ((int64_t)1 << 28)) continue;   // 1 GB of partial sums at most
            c.splits = (int)splits;
            c.per_split = (int)per;
            double us = div_up(c.full, slots) * kb * block_us;
            if (splits > 1) us += div_up(c.tail() * splits, slots) * per * block_us + 2.5 + (double)(splits * 8 + 2) * c.tail() * c.tile_elems() / 8.0e6;
            if (us < best_us) {
                best_us = us;
                best = c;
            }
        }
    }
    return best;
}

int64_t partial_bytes(const Cut& c) { return c.splits > 1 ? 4 * (int64_t)c.splits * c.tail() * c.tile_elems() : 0; }

template <int CG, int BN, int DT>
zero_status_t launch_shape(const GemmParams& P, int sms, cudaStream_t s)
{
    using S = GemmShape<CG, BN>;
    const cudaError_t set = allow_shared<gemm_kernel<CG, BN, DT>>(S::kSmem);
    if (set != cudaSuccess) return cuda_fail(set, "zero_linear: shared memory");
    const int64_t items = P.full + ((int64_t)P.tiles_m * P.tiles_n - P.full) * P.splits;
    const int grid = CG * (int)std::min<int64_t>(std::max(1, sms / CG), items);
    launch_after(gemm_kernel<CG, BN, DT>, grid, kGemmThreads, S::kSmem, s, P);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "zero_linear: launch");
}

// D = A B^T with epilogue E but for its split tiles, whose parts are left in `partial` (partial_bytes of
// it) and described in T; sum_tail ends them.
zero_status_t product(const Operand& a, const Operand& b, int dtype16, const Epilogue& E, float* partial, int sms, TailParams* T, cudaStream_t s)
{
    T->splits = 1;
    const int64_t M = a.rows, N = b.rows, K = a.inner;
    if (M == 0 || N == 0) return ZERO_OK;
    const bool bf = dtype16 == ZERO_BF16;
    if (K == 0) {
        const int grid = grid_of(M * N, sms, 8);
        if (bf) launch_after(empty_sum_kernel<ZERO_BF16>, grid, 256, 0, s, M, N, E);
        else launch_after(empty_sum_kernel<ZERO_FP16>, grid, 256, 0, s, M, N, E);
        const cudaError_t e = cudaGetLastError();
        return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "zero_linear: launch");
    }
    const Cut c = choose_cut(M, N, K);
    GemmParams P;
    // few rows: no zeros are copied for the rest, whose results are not stored
    P.a_rows = c.cg == 1 && !a.mn && M < kBM ? (int32_t)up(M, 8) : kBM;
    zero_status_t st = encode(&P.a, a, dtype16, P.a_rows, "zero_linear");
    if (st == ZERO_OK) st = encode(&P.b, b, dtype16, c.bn / c.cg, "zero_linear");
    if (st != ZERO_OK) return st;
    P.epi = E;
    P.partial = partial;
    P.M = (int32_t)M;
    P.N = (int32_t)N;
    P.k_blocks = (int32_t)div_up(K, kBK);
    P.full = (int32_t)c.full;
    P.splits = c.splits;
    P.k_per_split = c.per_split;
    P.tiles_m = (int32_t)c.tiles_m;
    P.tiles_n = (int32_t)c.tiles_n;
    P.a_mn = a.mn;
    P.b_mn = b.mn;
    P.rows_vec = (E.vec & kVecOut) && (!E.pre || (E.vec & kVecPre)) && (!E.residual || (E.vec & kVecRes));
    // fp32 accumulators; operand type; which operands lie along their rows; N / 8; M / 16
    P.idesc = (1u << 4) | ((bf ? 1u : 0u) << 7) | ((bf ? 1u : 0u) << 10) | ((a.mn ? 1u : 0u) << 15) |
              ((b.mn ? 1u : 0u) << 16) | ((uint32_t)(c.bn >> 3) << 17) | ((uint32_t)((kBM * c.cg) >> 4) << 24);
    if (c.cg == 2) st = bf ? launch_shape<2, 256, ZERO_BF16>(P, sms, s) : launch_shape<2, 256, ZERO_FP16>(P, sms, s);
    else if (c.bn == 128) st = bf ? launch_shape<1, 128, ZERO_BF16>(P, sms, s) : launch_shape<1, 128, ZERO_FP16>(P, sms, s);
    else st = bf ? launch_shape<1, 64, ZERO_BF16>(P, sms, s) : launch_shape<1, 64, ZERO_FP16>(P, sms, s);
    T->partial = partial;
    T->epi = E;
    T->M = P.M;
    T->N = P.N;
    T->full = P.full;
    T->splits = c.splits;
    T->tiles_m = P.tiles_m;
    T->tiles_n = P.tiles_n;
    T->tile_rows = kBM * c.cg;
    T->bn = c.bn;
    T->rows_vec = P.rows_vec;
    return st;
}

zero_status_t sum_tail(const TailParams& T, int dtype16, cudaStream_t s)
{
    if (T.splits == 1) return ZERO_OK;
    const dim3 grid((unsigned)(T.tile_rows / 8), (unsigned)(T.tiles_m * T.tiles_n - T.full));
    const cudaError_t e = dtype16 == ZERO_BF16 ? launch_after(tail_sum_kernel<ZERO_BF16>, grid, 256, 0, s, T)
                                               : launch_after(tail_sum_kernel<ZERO_FP16>, grid, 256, 0, s, T);
    return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "zero_linear: launch");
}

template <int DT, int ROWS>
zero_status_t launch_few(FewParams P, bool in_out, cudaStream_t s)
{
    cudaError_t e;
    if (!in_out) {
        // warps along K until there are sixteen an SM, by 256 elements in turn; the last shares may be short or
        // empty (K = 520 by four: 256, 256, 8 and none)
        const int64_t groups = div_up(P.N, kFewCols);
        P.split = 1;
        while (P.split < kFewWarps && groups * P.split < 16 * kGb300Sms && P.split * 256 < P.K) P.split *= 2;
        e = launch_after(few_rows_kernel<DT, ROWS>, (unsigned)div_up(groups, kFewWarps / P.split), 32 * kFewWarps, 0, s, P);
    } else {
        // as many parts of K as are resident at one time; each has at least 128 rows of W
        const int64_t blocks = div_up(P.N, 64);
        int parts = 1;
        while (parts < kFewParts && 2 * parts * blocks <= kFewResident * kGb300Sms && 256 * parts <= P.K) parts *= 2;
        e = launch_clusters_after(few_rows_deep_kernel<DT, ROWS>, dim3(1, parts), dim3((unsigned)blocks, parts), 32 * kFewDeep, 0, s, P);
    }
    return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "zero_linear: launch");
}

template <int DT>
zero_status_t launch_few(const FewParams& P, bool in_out, cudaStream_t s)
{
    return P.M == 1 ? launch_few<DT, 1>(P, in_out, s) : launch_few<DT, 2>(P, in_out, s);
}

// ------------------------------------------------------------------ host: the layer

constexpr int64_t kMaxSize = ZERO_LINEAR_MAX_SIZE;   // tile coordinates stay 32-bit

// How the dz pass is cut: threads across the columns (eight each) and workers a block, rows a worker.
// About eight blocks an SM where there are rows for them, and two rows a worker at least (the gradients of
// 777 x 1001 x 1603: 46.6 us, with four rows 49.3, with one 49.8).
struct DzCut {
    int tx = 256, ty = 1, chunk = 1;
    int64_t workers = 0;
};

DzCut dz_cut(int64_t rows, int64_t cols)
{
    DzCut c;
    while (c.tx > 32 && (int64_t)c.tx * 4 >= cols) c.tx /= 2;
    c.ty = 256 / c.tx;
    const int64_t across = std::max<int64_t>(1, div_up(cols, (int64_t)c.tx * 8));
    const int64_t want = std::max<int64_t>(1, 8 * kGb300Sms * c.ty / across);
    c.chunk = (int)std::max<int64_t>(2, div_up(std::max<int64_t>(rows, 1), want));
    c.workers = div_up(rows, c.chunk);
    return c;
}

// Everything a call needs, checked: strides filled in, and where its pieces lie in the workspace.
struct Layer {
    zero_linear_t a;
    bool bf = true;
    int64_t w_rows = 0, w_cols = 0;        // as stored
    bool copy_x = false, copy_w = false, make_dz = false, few = false;
    int64_t ld_x8 = 0, ld_w8 = 0, ld_dz = 0;
    int64_t at_x = 0, at_w = 0, at_dz = 0, at_sums = 0, at_partial = 0, at_partial_w = 0, bytes = 0;
    DzCut dz;
};

zero_status_t lay_out(const zero_linear_t* in, bool back, Layer* L, const char* who)
{
    const std::string w = std::string(who) + ": ";
    if (!in) return fail(ZERO_EINVAL, w + "NULL arguments");
    L->a = *in;
    zero_linear_t& a = L->a;
    if (a.rows < 0 || a.in_features < 0 || a.out_features < 0) return fail(ZERO_EINVAL, w + "negative size");
    if (a.rows > kMaxSize || a.in_features > kMaxSize || a.out_features > kMaxSize)
        return fail(ZERO_ERANGE, w + "a size beyond ZERO_LINEAR_MAX_SIZE");
    if (a.dtype16 != ZERO_BF16 && a.dtype16 != ZERO_FP16) return fail(ZERO_EINVAL, w + "bad dtype16");
    if (a.layout != ZERO_WEIGHT_OUT_IN && a.layout != ZERO_WEIGHT_IN_OUT) return fail(ZERO_EINVAL, w + "bad layout");
    if (a.activation < ZERO_ACT_NONE || a.activation > ZERO_ACT_SILU) return fail(ZERO_EINVAL, w + "bad activation");
    if (a.flags & ~(back ? ZERO_LINEAR_ACCUMULATE : 0)) return fail(ZERO_EINVAL, w + "unknown flag");
    L->bf = a.dtype16 == ZERO_BF16;
    L->w_rows = a.layout == ZERO_WEIGHT_OUT_IN ? a.out_features : a.in_features;
    L->w_cols = a.layout == ZERO_WEIGHT_OUT_IN ? a.in_features : a.out_features;
    struct {
        int64_t* ld;
        int64_t cols;
    } strides[] = {{&a.ld_x, a.in_features}, {&a.ld_w, L->w_cols},         {&a.ld_y, a.out_features},  {&a.ld_pre, a.out_features},
                   {&a.ld_residual, a.out_features}, {&a.ld_dy, a.out_features}, {&a.ld_dx, a.in_features}, {&a.ld_dw, L->w_cols}};
    for (auto& s : strides) {
        if (*s.ld == 0) *s.ld = s.cols;
        if (*s.ld < s.cols) return fail(ZERO_EINVAL, w + "a row stride is shorter than its row");
        if (*s.ld > ((int64_t)1 << 38)) return fail(ZERO_ERANGE, w + "a row stride beyond 2^38");
    }
    const void* every[] = {a.x, a.w, a.bias, a.residual, a.y, a.pre, a.dy, a.dx, a.dw, a.dbias};
    for (const void* p : every)
        if (!aligned(p, 2)) return fail(ZERO_EALIGN, w + "a pointer is not aligned to 2 bytes");
    const bool any_out = a.rows > 0 && a.out_features > 0;
    if (!back) {
        if (any_out && !a.y) return fail(ZERO_EINVAL, w + "y is NULL");
        if (any_out && a.in_features > 0 && (!a.x || !a.w)) return fail(ZERO_EINVAL, w + "x or w is NULL");
        if (any_out && a.residual == a.y && a.ld_residual != a.ld_y)
            return fail(ZERO_EINVAL, w + "y over residual needs its stride");
        if (any_out && a.pre && a.pre == a.y) return fail(ZERO_EINVAL, w + "pre and y are one buffer");
    } else {
        if (!a.dx && !a.dw && !a.dbias) return fail(ZERO_EINVAL, w + "no gradient asked for");
        if (any_out && !a.dy) return fail(ZERO_EINVAL, w + "dy is NULL");
        if (any_out && a.activation != ZERO_ACT_NONE && !a.pre) return fail(ZERO_EINVAL, w + "the activation's gradient needs pre");
        if (any_out && a.in_features > 0 && ((a.dx && !a.w) || (a.dw && !a.x)))
            return fail(ZERO_EINVAL, w + "x or w is NULL");
    }
    // the pieces of the workspace
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += up(bytes, 256);
        return here;
    };
    const bool use_x = back ? a.dw != nullptr : true, use_w = back ? a.dx != nullptr : true;
    const bool product_there = any_out && a.in_features > 0;
    L->ld_x8 = a.ld_x;
    L->ld_w8 = a.ld_w;
    L->ld_dz = a.ld_dy;
    L->few = !back && product_there && a.rows <= kFewRows && a.in_features % 8 == 0 && tma_ready(a.x, a.ld_x) && tma_ready(a.w, a.ld_w) &&
             (a.layout == ZERO_WEIGHT_OUT_IN || a.out_features % 8 == 0);
    L->copy_x = product_there && use_x && !L->few && !tma_ready(a.x, a.ld_x);
    L->copy_w = product_there && use_w && !L->few && !tma_ready(a.w, a.ld_w);
    if (L->copy_x) {
        L->ld_x8 = up(a.in_features, 8);
        L->at_x = take(2 * a.rows * L->ld_x8);
    }
    if (L->copy_w) {
        L->ld_w8 = up(L->w_cols, 8);
        L->at_w = take(2 * L->w_rows * L->ld_w8);
    }
    if (!back) {
        if (product_there && !L->few) L->at_partial = take(partial_bytes(choose_cut(a.rows, a.out_features, a.in_features)));
    } else {
        const bool products = product_there && (a.dx || a.dw);
        L->make_dz = products && (a.activation != ZERO_ACT_NONE || !tma_ready(a.dy, a.ld_dy));
        if (L->make_dz) {
            L->ld_dz = up(a.out_features, 8);
            L->at_dz = take(2 * a.rows * L->ld_dz);
        }
        L->dz = dz_cut(a.rows, a.out_features);
        if (a.dbias && any_out) L->at_sums = take(4 * L->dz.workers * up(a.out_features, 8));
        if (product_there && a.dx) L->at_partial = take(partial_bytes(choose_cut(a.rows, a.in_features, a.out_features)));
        if (product_there && a.dw) L->at_partial_w = take(partial_bytes(choose_cut(L->w_rows, L->w_cols, a.rows)));
    }
    L->bytes = at;
    return ZERO_OK;
}

zero_status_t check_workspace(const Layer& L, const void* workspace, int64_t bytes, const char* who)
{
    if (L.bytes == 0) return ZERO_OK;
    if (!workspace) return fail(ZERO_EINVAL, std::string(who) + ": workspace is NULL");
    if (!aligned(workspace, 16)) return fail(ZERO_EALIGN, std::string(who) + ": workspace not 16-byte aligned");
    if (bytes < L.bytes)
        return fail(ZERO_ERANGE, std::string(who) + ": workspace of " + std::to_string(bytes) + " bytes, " + std::to_string(L.bytes) + " needed");
    return ZERO_OK;
}

// The copies of x and w that the layer needs, into D; x and w become theirs.
void plan_copies(const Layer& L, char* ws, const void** x, const void** w, DzParams* D)
{
    std::memset(D, 0, sizeof(*D));
    auto job = [&](int i, const void** p, int64_t ld_src, int64_t at, int64_t ld, int64_t rows, int64_t cols) {
        AlignJob& J = D->copy[i];
        J.src = static_cast<const uint16_t*>(*p);
        J.dst = reinterpret_cast<uint16_t*>(ws + at);
        J.ld_src = ld_src;
        J.ld = ld;
        J.rows = rows;
        J.cols = cols;
        D->copy_blocks[i] = grid_of(rows * div_up(cols, 8), kGb300Sms, 8);
        *p = J.dst;
    };
    if (L.copy_x) job(0, x, L.a.ld_x, L.at_x, L.ld_x8, L.a.rows, L.a.in_features);
    if (L.copy_w) job(1, w, L.a.ld_w, L.at_w, L.ld_w8, L.w_rows, L.w_cols);
}

zero_status_t launch_dz(const Layer& L, const DzParams& D, cudaStream_t s)
{
    const int64_t blocks = (int64_t)D.dz_blocks + D.copy_blocks[0] + D.copy_blocks[1];
    if (blocks == 0) return ZERO_OK;
    const dim3 threads(L.dz.tx, L.dz.ty);
    if (L.bf) launch_after(dz_kernel<ZERO_BF16>, (unsigned)blocks, threads, 0, s, D);
    else launch_after(dz_kernel<ZERO_FP16>, (unsigned)blocks, threads, 0, s, D);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "zero_linear: launch");
}

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" {

zero_status_t zero_linear_workspace(const zero_linear_t* a, int backward, int64_t* bytes)
try {
    if (!bytes) return fail(ZERO_EINVAL, "zero_linear_workspace: NULL argument");
    Layer L;
    const zero_status_t st = lay_out(a, backward != 0, &L, "zero_linear_workspace");
    if (st == ZERO_OK) *bytes = L.bytes;
    return st;
}
catch (...) {
    return exception_status("zero_linear_workspace");
}

zero_status_t zero_linear(const zero_linear_t* args, void* workspace, int64_t workspace_bytes, void* stream)
try {
    Layer L;
    zero_status_t st = lay_out(args, false, &L, "zero_linear");
    if (st == ZERO_OK) st = check_workspace(L, workspace, workspace_bytes, "zero_linear");
    if (st != ZERO_OK) return st;
    const zero_linear_t& a = L.a;
    if (a.rows == 0 || a.out_features == 0) return ZERO_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    const void *x = a.x, *w = a.w;
    if (L.copy_x || L.copy_w) {
        DzParams D;
        plan_copies(L, ws, &x, &w, &D);
        st = launch_dz(L, D, s);
        if (st != ZERO_OK) return st;
    }
    Epilogue E;
    E.out = static_cast<uint16_t*>(a.y);
    E.pre = static_cast<uint16_t*>(a.pre);
    E.bias = static_cast<const uint16_t*>(a.bias);
    E.residual = static_cast<const uint16_t*>(a.residual);
    E.ld_out = a.ld_y;
    E.ld_pre = a.ld_pre;
    E.ld_res = a.ld_residual;
    E.act = a.activation;
    E.vec = vec_flag(a.y, a.ld_y, kVecOut) | vec_flag(a.pre, a.ld_pre, kVecPre) |
            vec_flag(a.residual, a.ld_residual, kVecRes) | vec_flag(a.bias, 0, kVecBias);
    if (L.few) {
        FewParams P;
        P.x = static_cast<const uint16_t*>(a.x);
        P.w = static_cast<const uint16_t*>(a.w);
        P.epi = E;
        P.ld_x = a.ld_x;
        P.ld_w = a.ld_w;
        P.M = (int32_t)a.rows;
        P.N = (int32_t)a.out_features;
        P.K = (int32_t)a.in_features;
        const bool in_out = a.layout == ZERO_WEIGHT_IN_OUT;
        return L.bf ? launch_few<ZERO_BF16>(P, in_out, s) : launch_few<ZERO_FP16>(P, in_out, s);
    }
    const Operand A{x, a.rows, a.in_features, L.ld_x8, false};
    const Operand B{w, a.out_features, a.in_features, L.ld_w8, a.layout == ZERO_WEIGHT_IN_OUT};
    TailParams T;
    st = product(A, B, a.dtype16, E, reinterpret_cast<float*>(ws + L.at_partial), kGb300Sms, &T, s);
    return st == ZERO_OK ? sum_tail(T, a.dtype16, s) : st;
}
catch (...) {
    return exception_status("zero_linear");
}

zero_status_t zero_linear_backward(const zero_linear_t* args, void* workspace, int64_t workspace_bytes, void* stream)
try {
    Layer L;
    zero_status_t st = lay_out(args, true, &L, "zero_linear_backward");
    if (st == ZERO_OK) st = check_workspace(L, workspace, workspace_bytes, "zero_linear_backward");
    if (st != ZERO_OK) return st;
    const zero_linear_t& a = L.a;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    const bool accumulate = a.flags & ZERO_LINEAR_ACCUMULATE, any_out = a.rows > 0 && a.out_features > 0;
    const void *x = a.x, *w = a.w, *dz = a.dy;
    DzParams D;
    plan_copies(L, ws, &x, &w, &D);
    float* sums = a.dbias && any_out ? reinterpret_cast<float*>(ws + L.at_sums) : nullptr;
    if (L.make_dz || sums) {
        D.dy = static_cast<const uint16_t*>(a.dy);
        D.pre = a.activation != ZERO_ACT_NONE ? static_cast<const uint16_t*>(a.pre) : nullptr;
        D.dz = L.make_dz ? reinterpret_cast<uint16_t*>(ws + L.at_dz) : nullptr;
        D.sums = sums;
        D.rows = a.rows;
        D.cols = a.out_features;
        D.ld_dy = a.ld_dy;
        D.ld_pre = a.ld_pre;
        D.ld_dz = up(a.out_features, 8);
        D.act = a.activation;
        D.vec_dy = vec_flag(a.dy, a.ld_dy, 1);
        D.vec_pre = vec_flag(a.pre, a.ld_pre, 1);
        D.chunk = L.dz.chunk;
        D.across = (int32_t)div_up(a.out_features, (int64_t)L.dz.tx * 8);
        D.dz_blocks = (int32_t)(D.across * div_up(L.dz.workers, L.dz.ty));
        if (L.make_dz) dz = D.dz;
    }
    st = launch_dz(L, D, s);
    if (st != ZERO_OK) return st;
    // The column sums and dx need dz and not one another, nor does dw need them; but each waits for the one
    // before it, as only a kernel's own wait makes what was written before the call, or by its first launch,
    // visible to it.  Both products' split tiles are summed at the end.
    if (a.dbias && a.out_features > 0 && !(a.rows == 0 && accumulate)) {
        const unsigned grid = (unsigned)div_up(a.out_features, 32);
        const dim3 threads(32, 8);
        const int64_t workers = any_out ? L.dz.workers : 0;
        uint16_t* db = static_cast<uint16_t*>(a.dbias);
        if (L.bf) launch_after(column_sum_kernel<ZERO_BF16>, grid, threads, 0, s, sums, up(a.out_features, 8), workers, a.out_features, db, accumulate);
        else launch_after(column_sum_kernel<ZERO_FP16>, grid, threads, 0, s, sums, up(a.out_features, 8), workers, a.out_features, db, accumulate);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "zero_linear_backward: launch");
    TailParams Tx, Tw;
    Tx.splits = Tw.splits = 1;
    Epilogue E;
    std::memset(&E, 0, sizeof(E));
    E.act = ZERO_ACT_NONE;
    if (a.dx) {
        E.out = static_cast<uint16_t*>(a.dx);
        E.ld_out = a.ld_dx;
        E.vec = vec_flag(a.dx, a.ld_dx, kVecOut);
        const Operand A{dz, a.rows, a.out_features, L.ld_dz, false};
        const Operand B{w, a.in_features, a.out_features, L.ld_w8, a.layout == ZERO_WEIGHT_OUT_IN};
        st = product(A, B, a.dtype16, E, reinterpret_cast<float*>(ws + L.at_partial), kGb300Sms, &Tx, s);
        if (st != ZERO_OK) return st;
    }
    if (a.dw && !(a.rows == 0 && accumulate)) {
        E.out = static_cast<uint16_t*>(a.dw);
        E.ld_out = a.ld_dw;
        E.residual = accumulate ? E.out : nullptr;
        E.ld_res = a.ld_dw;
        E.vec = vec_flag(a.dw, a.ld_dw, kVecOut | kVecRes);
        const Operand X{x, a.in_features, a.rows, L.ld_x8, true}, Z{dz, a.out_features, a.rows, L.ld_dz, true};
        const bool out_in = a.layout == ZERO_WEIGHT_OUT_IN;
        st = product(out_in ? Z : X, out_in ? X : Z, a.dtype16, E, reinterpret_cast<float*>(ws + L.at_partial_w), kGb300Sms, &Tw, s);
        if (st != ZERO_OK) return st;
    }
    st = sum_tail(Tx, a.dtype16, s);
    return st == ZERO_OK ? sum_tail(Tw, a.dtype16, s) : st;
}
catch (...) {
    return exception_status("zero_linear_backward");
}

zero_status_t zero_operators_check(void* stream)
try {
    uint32_t linear = 0, norm = 0, gated = 0, muon = 0;
    cudaError_t e = take_error_word(g_linear_error, &linear, static_cast<cudaStream_t>(stream));
    if (e == cudaSuccess) e = take_norm_error(&norm, stream);
    if (e == cudaSuccess) e = take_gated_error(&gated, stream);
    if (e == cudaSuccess) e = take_muon_error(&muon, stream);
    if (e != cudaSuccess) return cuda_fail(e, "zero_operators_check");
    if (!linear && !norm && !gated && !muon) return ZERO_OK;
    return fail(ZERO_ETIMEOUT, std::string(linear ? "zero_linear" : norm ? "zero_block_norm" : gated ? "zero_gated" : "zero_muon") +
                                   ": a bounded wait ran out; outputs since the last check are not final");
}
catch (...) {
    return exception_status("zero_operators_check");
}

}  // extern "C"
