// zero_gated.cu -- the first half of a gated feed-forward block, forward and backward (zero_gated_*):
//   g = x Wg + bg, u = x Wu + bu, h = act(g) * u
//   dg = dh u act'(g), du = dh act(g);  dx = dg Wg^T + du Wu^T;  dWg = x^T dg, dWu = x^T du;  db = column sums
//
// Both projections are one product on the tensor cores: half of a tile's columns are Wg's and half Wu's, at the same
// place, so that x is staged once for both and a thread of the epilogue holds g and u of the same elements; h leaves
// it without g and u having been to memory (they are written where the gradients will want them).  dx is one product
// too, its inner dimension Wg's columns and then Wu's; its tiles, those of the weights' two gradients and the sums of
// the biases' are one launch, so that no round of tiles has to be full.  dg and du are formed by a pass of their own, as
// the products need them in two layouts and the biases their sums.  Where there are few tiles and a long inner
// dimension, parts of it are tiles of their own, summed in order by the warp that ends last.
//
// Measured on one GB300 (cuBLAS bf16: 1,939 TFLOP/s in a burst, 1,731 sustained under the power cap): 8192 tokens
// 4096 -> 11008 with g and u kept 825 to 888 us, 1,660 to 1,790 TFLOP/s; their gradients 1,853 to 1,966, of which 133 are dg
// and du (HBM); 2048 tokens 2048 -> 8192 192 to 197 (dg and du 26, the rest 145 alone, tensor cores busy 89 %); 777 tokens
// 1001 -> 1603, every row off the 16-byte grid, 36; one token 4096 -> 11008 29.5 (6.1 TB/s), 24 tokens 2048 -> 8192
// 14.7.  Tiles of few inner blocks are bound by their ends: 256 x 256 take 5 us with g and u kept, as long as 16 blocks.
#include <cmath>
#include <cstring>

#include "zero_mma.cuh"

namespace zero {
namespace {

// Set by a kernel whose bounded wait ran out (zero_operators_check reads and clears it).
__device__ uint32_t g_gated_error;

// What a launch's tiles are.
enum { kForward = 0, kBackward = 1 };   // g and u; dx, then dWg and dWu

// One product of the backward pass.  dx (the first): a and b of both pairs, its inner blocks of the first and then the
// second; a weight's gradient: the first of each.
struct Product {
    CUtensorMap a[2], b[2];
    Matrix16 out;
    int32_t tiles_m, tiles_n, k_blocks, k_first;
    int32_t splits, k_per_split; // parts of the inner dimension, and the inner blocks of one (the last may have fewer)
    int32_t tile0, part0;        // of the products in parts: the tiles, and the parts, before this product's
    int32_t a_mn, b_mn;          // operand stored along its own rows instead of along K
    uint32_t idesc;
};

// Tiles of two kinds dealt to w workers: every w-th of n1, then of n2 `more` to each of the first `ahead` workers (those
// with one of the first kind more) and `rest` to each of the others, as even as that goes.
struct Deal {
    int32_t n1, n2, w, ahead, more, rest;
};

template <int MODE>
struct GatedParams {
    Product part[MODE == kForward ? 1 : 3];   // forward: x, Wg and Wu (a[0], b[0], b[1]); backward: dx, dWg, dWu, those that are there
    Matrix16 out[3];             // forward: h, g, u (p NULL: not kept)
    const uint16_t* bias[2];     // forward: of g and u, or NULL
    Deal deal;                   // parts counted each.  Forward: n1 whole tiles, n2 parts of the others; backward: dx's (part[0]), the others'
    float4* partial;             // a part's sums: [tile][part][warp][..]
    uint32_t* tickets;           // [tile][warp]: parts that are there; 0 at first
    int32_t parts_at;            // backward: the first part that is a weight's gradient: 1 after dx, or 0
    int32_t a_rows;              // rows of A that a copy brings (kBM, or fewer where A has no more)
    int32_t act, accumulate, bias_vec;
    // backward: the biases' gradients from the sums of `workers` workers, [worker][2][ld]
    const float* sums;
    uint16_t* db[2];
    int64_t ld, workers, cols;
};

// g becomes act(g) u.
template <int ACT>
__device__ __forceinline__ void gate_each(float (&g)[32], const float (&u)[32])
{
#pragma unroll
    for (int j = 0; j < 32; ++j) g[j] = act_value(g[j], ACT) * u[j];
}

__device__ __forceinline__ void gate_values(float (&g)[32], const float (&u)[32], int act)
{
    switch (act) {
    case ZERO_ACT_RELU: gate_each<ZERO_ACT_RELU>(g, u); break;
    case ZERO_ACT_GELU_TANH: gate_each<ZERO_ACT_GELU_TANH>(g, u); break;
    case ZERO_ACT_GELU: gate_each<ZERO_ACT_GELU>(g, u); break;
    case ZERO_ACT_SILU: gate_each<ZERO_ACT_SILU>(g, u); break;
    default: gate_each<ZERO_ACT_NONE>(g, u);
    }
}

// 32 columns of a bias from col0 on, packed; zeros past the last and without one.
__device__ __forceinline__ void fetch_bias(uint4 (&v)[4], const uint16_t* bias, bool vec, int64_t col0, int64_t cols)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = bias ? (int)max((int64_t)0, min((int64_t)8, cols - col0 - 8 * i)) : 0;
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (n == 8 && vec) {
            v[i] = *reinterpret_cast<const uint4*>(bias + col0 + 8 * i);
        } else if (n > 0) {
            const uint16_t* p = bias + col0 + 8 * i;
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = (2 * j < n ? p[2 * j] : 0u) | ((2 * j + 1 < n ? (uint32_t)p[2 * j + 1] : 0u) << 16);
            v[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

template <int DT>
__device__ __forceinline__ void add_bias(float (&x)[32], const uint4 (&v)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float a, b;
            widen2<DT>(word(v[i], j), a, b);
            x[8 * i + 2 * j] += a;
            x[8 * i + 2 * j + 1] += b;
        }
}

// Sums over the workers of 32 columns from c0 on, by a warp: eight lanes of four columns each, each eight a quarter of
// the workers, in a fixed order.
template <int DT>
__device__ __forceinline__ void add_workers(const float* sums, int64_t ld, int64_t workers, int64_t c0, int64_t cols, uint16_t* out, int accumulate, int lane)
{
    if (!out) return;
    const int64_t c = c0 + (lane & 7) * 4;
    const bool mine = c < cols;                  // rows of a multiple of eight: four columns are there, or none
    float4 s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int64_t w = lane >> 3; mine && w < workers; w += 32) {
        float4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = w + 4 * j < workers ? *reinterpret_cast<const float4*>(sums + (w + 4 * j) * 2 * ld + c) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s[j & 3].x += v[j].x;
            s[j & 3].y += v[j].y;
            s[j & 3].z += v[j].z;
            s[j & 3].w += v[j].w;
        }
    }
    float x[4] = {(s[0].x + s[1].x) + (s[2].x + s[3].x), (s[0].y + s[1].y) + (s[2].y + s[3].y), (s[0].z + s[1].z) + (s[2].z + s[3].z),
                  (s[0].w + s[1].w) + (s[2].w + s[3].w)};
#pragma unroll
    for (int o = 8; o < 32; o *= 2)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] += __shfl_xor_sync(0xFFFFFFFFu, x[j], o);
    if (lane >= 8) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (c + j >= cols) break;
        if (accumulate) x[j] += widen1<DT>(out[c + j]);
        out[c + j] = narrow1<DT>(x[j]);
    }
}

template <int CG, int BN, int MODE, int DT>
struct GatedWork {
    const GatedParams<MODE>& P;
    static constexpr int kBRows = BN / CG;
    struct Item {
        int m, n, kb, part;
        int splits, k0, slice, tile;   // parts of the tile; the first inner block; which part; its tile among those in parts
    };
    // The biases of a tile's first part are loaded while its products run.
    struct Ahead {
        uint4 bias[MODE == kForward ? 2 : 1][4];
    };
    __device__ __forceinline__ void biases(const Item& I, int c, Ahead& A) const
    {
        if constexpr (MODE == kForward) {
            const int64_t col0 = (int64_t)I.n * (BN / 2) + c;
            fetch_bias(A.bias[0], P.bias[0], P.bias_vec & 1, col0, P.out[0].cols);
            fetch_bias(A.bias[1], P.bias[1], P.bias_vec & 2, col0, P.out[0].cols);
        }
    }
    __device__ __forceinline__ void prepare(const Item& I, int, int half, int, int, Ahead& A) const
    {
        if (P.bias[0] || P.bias[1]) biases(I, half * kEpiCols, A);
    }
    static constexpr bool kScout = false;
    __device__ __forceinline__ void done(const Item&) const {}
    __device__ __forceinline__ void gave_up() const {}

    __device__ __forceinline__ void range(int worker, int, int& i, int& end, int& step) const
    {
        const Deal& D = P.deal;
        if constexpr (MODE == kForward) {
            // in turn: the tiles of the first kind are whole rounds, or all there are
            i = worker;
            step = D.w;
            end = D.n1 + D.n2;
        } else {
            i = 0;
            step = 1;
            end = worker < D.n1 ? (D.n1 - worker + D.w - 1) / D.w : 0;
            // of the second kind: the places that it has, up to the last tile
            const int first = worker < D.ahead ? worker : D.ahead * D.more + worker - D.ahead;
            const int stride = worker < D.ahead ? D.ahead : D.w - D.ahead, most = worker < D.ahead ? D.more : D.rest;
            if (first < D.n2) end += min(most, (D.n2 - first + stride - 1) / stride);
        }
    }

    __device__ __forceinline__ Item item(int i) const
    {
        const Deal& D = P.deal;
        Item I;
        I.part = 0;
        int tile, splits = P.part[0].splits;
        if constexpr (MODE == kForward) {
            tile = i;
            if (i < D.n1) splits = 1;
            else tile -= D.n1;
        } else {
            const int worker = blockIdx.x / CG;
            tile = worker + i * D.w;
            if (tile >= D.n1) {
                const int n1 = worker < D.n1 ? (D.n1 - worker + D.w - 1) / D.w : 0, stride = worker < D.ahead ? D.ahead : D.w - D.ahead;
                tile = (worker < D.ahead ? worker : D.ahead * D.more + worker - D.ahead) + (i - n1) * stride;
                I.part = P.parts_at;
                const int per = P.part[I.part].tiles_m * P.part[I.part].tiles_n * P.part[I.part].splits;
                if (tile >= per) {
                    tile -= per;
                    ++I.part;
                }
                splits = P.part[I.part].splits;
            }
        }
        const Product& Q = P.part[I.part];
        I.splits = splits;
        I.slice = 0;
        I.kb = Q.k_blocks;
        if (splits > 1) {
            I.slice = tile % splits;
            tile /= splits;
            I.kb = min(Q.k_blocks - I.slice * Q.k_per_split, Q.k_per_split);
        }
        I.k0 = I.slice * Q.k_per_split;
        I.tile = Q.tile0 + tile;
        if (MODE == kForward && i >= D.n1) tile += D.n1;
        tile_at(Q.tiles_m, Q.tiles_n, tile, I.m, I.n);
        return I;
    }
    __device__ __forceinline__ uint32_t bytes(const Item& I) const { return CG * ((P.part[I.part].a_mn ? kBM : P.a_rows) + kBRows) * (kBK * 2); }
    __device__ __forceinline__ bool a_mn(const Item& I, int) const { return P.part[I.part].a_mn; }
    __device__ __forceinline__ bool b_mn(const Item& I, int) const { return P.part[I.part].b_mn; }
    __device__ __forceinline__ uint32_t idesc(const Item& I, int) const { return P.part[I.part].idesc; }

    // ROWS rows of an operand: along K in one box, along its own rows in boxes of 64
    template <int ROWS>
    __device__ __forceinline__ static void bring(const CUtensorMap* map, bool mn, uint32_t at, int row, int k, uint32_t bar)
    {
        if (mn) {
#pragma unroll
            for (int i = 0; i < ROWS / 64; ++i) tma_load_2d<CG>(at + i * (kBK * 128), map, row + 64 * i, k, bar);
        } else {
            tma_load_2d<CG>(at, map, k, row, bar);
        }
    }

    __device__ __forceinline__ void load(const Item& I, int kb, uint32_t a, uint32_t b, uint32_t bar, int rank) const
    {
        const Product& Q = P.part[I.part];
        const int row_a = (I.m * CG + rank) * kBM;
        kb += I.k0;
        if constexpr (MODE == kForward) {
            const int k = kb * kBK;
            bring<kBM>(&Q.a[0], false, a, row_a, k, bar);
            if constexpr (CG == 2) {
                // the pair's first block brings Wg's half of the columns and the second Wu's
                bring<kBRows>(&Q.b[rank], Q.b_mn, b, I.n * kBRows, k, bar);
            } else {
                for (int i = 0; i < 2; ++i) bring<64>(&Q.b[i], Q.b_mn, b + i * (64 * kBK * 2), I.n * 64, k, bar);
            }
        } else {
            const bool second = kb >= Q.k_first;
            const int pair = second ? 1 : 0, k = (second ? kb - Q.k_first : kb) * kBK;
            bring<kBM>(&Q.a[pair], Q.a_mn, a, row_a, k, bar);
            bring<kBRows>(&Q.b[pair], Q.b_mn, b, I.n * BN + rank * kBRows, k, bar);
        }
    }

    // The biases' gradients: 32 columns of one of them a warp, four a lane and every fourth worker; the workers' sums in
    // a fixed order, in fp32.
    __device__ __forceinline__ void aside(int lane) const
    {
        if constexpr (MODE == kBackward) {
            if (!P.sums) return;
            const int64_t parts = (P.cols + 31) / 32;
            for (int64_t i = blockIdx.x; i < 2 * parts; i += gridDim.x) {
                const int which = i >= parts;
                add_workers<DT>(P.sums + which * P.ld, P.ld, P.workers, (i - which * parts) * 32, P.cols, P.db[which], P.accumulate, lane);
            }
        }
    }

    // ---- a tile's end
    static constexpr int kParts = BN / 64;                     // 32 x 32 results of a warp
    static constexpr int kWidth = MODE == kForward ? BN / 2 : BN;   // columns of the result

    // Where this warp's sums of part `slice` are: kParts of eight rows of 16 bytes a lane.
    __device__ __forceinline__ float4* sums_at(const Item& I, int slice, int warp, int rank) const
    {
        const Product& Q = P.part[I.part];
        const int64_t part = Q.part0 + (int64_t)(I.tile - Q.tile0) * I.splits + slice;
        return P.partial + ((part * CG + rank) * kEpiWarps + warp) * (kParts * 8 * 32);
    }

    // The warp's results are kept beside the other parts'; is it the last of them?
    __device__ __forceinline__ bool keep_part(const Item& I, uint32_t acc, int half, int warp, int rank, int lane) const
    {
        float4* q = sums_at(I, I.slice, warp, rank) + lane;
        for (int c = half * kEpiCols; c < kWidth; c += 2 * kEpiCols)
            for (int k = 0; k < (MODE == kForward ? 2 : 1); ++k) {
                float x[32];
                tmem_load32(acc + k * kWidth + c, x);
#pragma unroll
                for (int j = 0; j < 8; ++j) __stcg(q + j * 32, make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]));
                q += 8 * 32;
            }
        __threadfence();
        __syncwarp();
        uint32_t before = 0;
        if (lane == 0) before = atomicAdd(P.tickets + ((int64_t)I.tile * CG + rank) * kEpiWarps + warp, 1u);
        before = __shfl_sync(0xFFFFFFFFu, before, 0);
        __threadfence();
        return before == (uint32_t)I.splits - 1;
    }

    // Results `part` of the warp: from TMEM, or the sum of all parts.
    __device__ __forceinline__ void results(const Item& I, uint32_t at, int part, int warp, int rank, int lane, float (&x)[32]) const
    {
        if (I.splits == 1) {
            tmem_load32(at, x);
            return;
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = 0.0f;
        const float4* q = sums_at(I, 0, warp, rank) + part * (8 * 32) + lane;
        const int64_t next = (int64_t)CG * kEpiWarps * (kParts * 8 * 32);
        auto add = [&](const float4 (&v)[8]) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[4 * j] += v[j].x;
                x[4 * j + 1] += v[j].y;
                x[4 * j + 2] += v[j].z;
                x[4 * j + 3] += v[j].w;
            }
        };
        // in order, two at a time: what a part costs is the way to L2
        int s = 0;
        for (; s + 2 <= I.splits; s += 2, q += 2 * next) {
            float4 v[8], w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __ldcg(q + j * 32);
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = __ldcg(q + next + j * 32);
            add(v);
            add(w);
        }
        if (s < I.splits) {
            float4 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __ldcg(q + j * 32);
            add(v);
        }
    }

    __device__ __forceinline__ void finish(const Item& I, Ahead& A, uint32_t acc, int quad, int half, uint32_t stage, int rank, int lane) const
    {
        const int64_t row0 = ((int64_t)I.m * CG + rank) * kBM + quad * 32;
        const int warp = quad + 4 * half;
        if (row0 >= (MODE == kForward ? P.out[0].rows : P.part[I.part].out.rows)) return;
        if (I.splits > 1 && !keep_part(I, acc, half, warp, rank, lane)) return;
        int part = 0;
        if constexpr (MODE == kForward) {
            const Matrix16& H = P.out[0];
            for (int c = half * kEpiCols; c < kWidth; c += 2 * kEpiCols, part += 2) {
                const int64_t col0 = (int64_t)I.n * kWidth + c;
                if (col0 >= H.cols) break;
                float g[32], u[32];
                results(I, acc + c, part, warp, rank, lane, g);
                results(I, acc + kWidth + c, part + 1, warp, rank, lane, u);
                if (P.bias[0] || P.bias[1]) {
                    add_bias<DT>(g, A.bias[0]);
                    add_bias<DT>(u, A.bias[1]);
                    if (c + 2 * kEpiCols < kWidth) biases(I, c + 2 * kEpiCols, A);
                }
                if (P.out[1].p) put_tile<DT>(stage, lane, g, P.out[1], row0, col0);
                if (P.out[2].p) put_tile<DT>(stage + kTile16Bytes, lane, u, P.out[2], row0, col0);
                gate_values(g, u, P.act);
                put_tile<DT>(stage, lane, g, H, row0, col0);
            }
        } else {
            const Product& Q = P.part[I.part];
            const Matrix16& D = Q.out;
            const bool add = P.accumulate && I.part >= P.parts_at;
            for (int c = half * kEpiCols; c < kWidth; c += 2 * kEpiCols, ++part) {
                const int64_t col0 = (int64_t)I.n * BN + c;
                if (col0 >= D.cols) break;
                float x[32];
                results(I, acc + c, part, warp, rank, lane, x);
                if (add) add_tile<DT>(stage + kTile16Bytes, lane, 1.0f, x, D, row0, col0);
                // of few rows, the weights' gradients are little but this: 128 tokens, 4096 -> 11008, 73 -> 62 us for both
                put_tile<DT, true>(stage, lane, x, D, row0, col0);
            }
        }
    }
};

template <int CG, int BN, int MODE, int DT>
__global__ void __cluster_dims__(CG, 1, 1) __launch_bounds__(kGemmThreads, 1) gated_kernel(const __grid_constant__ GatedParams<MODE> P)
{
    extern __shared__ unsigned char smem_raw[];
    Tiles<CG, BN> T;
    T.open(smem_raw);
    after_earlier_work();
    T.run(GatedWork<CG, BN, MODE, DT>{P}, &g_gated_error);
}

// The block over an empty inner dimension: g = bg, u = bu.
template <int DT>
__global__ void __launch_bounds__(256) gated_empty_kernel(const __grid_constant__ GatedParams<kForward> P)
{
    after_earlier_work();
    const Matrix16 &H = P.out[0], &G = P.out[1], &U = P.out[2];
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < H.rows * H.cols; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / H.cols, col = i - row * H.cols;
        const float g = P.bias[0] ? widen1<DT>(P.bias[0][col]) : 0.0f, u = P.bias[1] ? widen1<DT>(P.bias[1][col]) : 0.0f;
        if (G.p) G.p[row * G.ld + col] = narrow1<DT>(g);
        if (U.p) U.p[row * U.ld + col] = narrow1<DT>(u);
        H.p[row * H.ld + col] = narrow1<DT>(act_value(g, P.act) * u);
    }
}

// ------------------------------------------------------------------ dg and du, and aligned copies

// What precedes the products, one launch: dg and du with their column sums, and the copies of x and the weights.
struct SplitParams {
    AlignJob copy[3];
    int32_t blocks, across;      // blocks of the pass, and how many of them share rows
    int32_t copy_blocks[3];
    const uint16_t *dh, *gate, *up;
    uint16_t *dg, *du;           // rows of ld elements, 16-byte aligned; NULL: only the sums
    float* sums;                 // [block of workers][2][ld] column sums, or NULL
    uint32_t* tickets;           // set to 0
    int32_t n_tickets;
    int64_t rows, cols, ld_dh, ld_gate, ld_up, ld;
    int32_t act, vec, chunk;     // vec: every row starts on 16 bytes; chunk: consecutive rows a worker takes
};

template <int ACT>
__device__ __forceinline__ void split_each(const float (&d)[8], float (&g)[8], float (&u)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float a = act_value(g[j], ACT), s = act_slope(g[j], ACT), up = u[j];
        u[j] = d[j] * a;
        // the slope, at most 1.2, before dh: dh u alone may leave fp32's range in bf16 (and a slope of 0 then made it NaN)
        g[j] = d[j] * (up * s);
    }
}

// g and u become dg and du.
__device__ __forceinline__ void split_values(const float (&d)[8], float (&g)[8], float (&u)[8], int act)
{
    switch (act) {
    case ZERO_ACT_RELU: split_each<ZERO_ACT_RELU>(d, g, u); break;
    case ZERO_ACT_GELU_TANH: split_each<ZERO_ACT_GELU_TANH>(d, g, u); break;
    case ZERO_ACT_GELU: split_each<ZERO_ACT_GELU>(d, g, u); break;
    case ZERO_ACT_SILU: split_each<ZERO_ACT_SILU>(d, g, u); break;
    default: split_each<ZERO_ACT_NONE>(d, g, u);
    }
}

template <int DT>
__device__ __forceinline__ void widen8(const uint4& w, float (&x)[8])
{
    widen2<DT>(w.x, x[0], x[1]);
    widen2<DT>(w.y, x[2], x[3]);
    widen2<DT>(w.z, x[4], x[5]);
    widen2<DT>(w.w, x[6], x[7]);
}

// FULL: all eight columns are there, by 16-byte accesses; else `n` of them, and zeros.
template <bool FULL>
__device__ __forceinline__ uint4 fetch8(const uint16_t* p, int n)
{
    if constexpr (FULL) {
        return __ldcs(reinterpret_cast<const uint4*>(p));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = (2 * j < n ? p[2 * j] : 0u) | ((2 * j + 1 < n ? (uint32_t)p[2 * j + 1] : 0u) << 16);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <int DT, bool FULL, int FLIGHT>
__device__ __forceinline__ void split_rows(const SplitParams& P, int64_t col, int n, int64_t r, float (&sg)[8], float (&su)[8])
{
    uint4 d[FLIGHT], g[FLIGHT], u[FLIGHT];
#pragma unroll
    for (int i = 0; i < FLIGHT; ++i) {
        d[i] = fetch8<FULL>(P.dh + (r + i) * P.ld_dh + col, n);
        g[i] = fetch8<FULL>(P.gate + (r + i) * P.ld_gate + col, n);
        u[i] = fetch8<FULL>(P.up + (r + i) * P.ld_up + col, n);
    }
#pragma unroll
    for (int i = 0; i < FLIGHT; ++i) {
        float x[8], y[8], z[8];
        widen8<DT>(d[i], x);
        widen8<DT>(g[i], y);
        widen8<DT>(u[i], z);
        split_values(x, y, z, P.act);
        if (P.sums) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sg[j] += FULL || j < n ? y[j] : 0.0f;
                su[j] += FULL || j < n ? z[j] : 0.0f;
            }
        }
        if (P.dg) {
            store8<DT>(P.dg + (r + i) * P.ld + col, true, 8, y);      // rows of a multiple of 8
            store8<DT>(P.du + (r + i) * P.ld + col, true, 8, z);
        }
    }
}

// Rows copied to rows that start on 16 bytes, by block b of n: kCopies times eight elements a thread, all loaded before
// any is stored.
constexpr int kCopies = 2;

__device__ __forceinline__ void copy_rows(const AlignJob& J, int b, int n, int thread)
{
    const int64_t per_row = (J.cols + 7) / 8, total = J.rows * per_row, step = (int64_t)n * 256;
    for (int64_t i0 = (int64_t)b * 256 + thread; i0 < total; i0 += kCopies * step) {
        uint4 v[kCopies];
        int64_t to[kCopies];
#pragma unroll
        for (int k = 0; k < kCopies; ++k) {
            const int64_t i = i0 + k * step, row = total < INT32_MAX ? (int64_t)((uint32_t)i / (uint32_t)per_row) : i / per_row, col = (i - row * per_row) * 8;
            to[k] = row * J.ld + col;
            v[k] = i < total ? fetch8<false>(J.src + row * J.ld_src + col, (int)min((int64_t)8, J.cols - col)) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int k = 0; k < kCopies; ++k)
            if (i0 + k * step < total) *reinterpret_cast<uint4*>(J.dst + to[k]) = v[k];
    }
}

// A thread takes eight columns of a worker's rows (blocks of up to 2048 columns; narrower ones hold several
// workers), so that the sums need no exchange.
template <int DT>
__global__ void __launch_bounds__(256, 3) split_kernel(const __grid_constant__ SplitParams P)
{
    after_earlier_work();
    constexpr int kFlight = 2;
    __shared__ float4 turned[256][4];
    const int thread = threadIdx.y * blockDim.x + threadIdx.x;
    for (int i = blockIdx.x * 256 + thread; i < P.n_tickets; i += gridDim.x * 256) P.tickets[i] = 0;
    if ((int)blockIdx.x >= P.blocks) {
        int b = blockIdx.x - P.blocks, which = 0;
        while (b >= P.copy_blocks[which]) b -= P.copy_blocks[which++];
        copy_rows(P.copy[which], b, P.copy_blocks[which], thread);
        return;
    }
    const int by = blockIdx.x / P.across, bx = blockIdx.x - by * P.across;
    const int64_t col = ((int64_t)bx * blockDim.x + threadIdx.x) * 8;
    const int n = (int)max((int64_t)0, min((int64_t)8, P.cols - col));
    const int64_t worker = (int64_t)by * blockDim.y + threadIdx.y;
    const int64_t r1 = min(P.rows, (worker + 1) * P.chunk);
    int64_t r = worker * P.chunk;
    float sg[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f}, su[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (n == 8 && P.vec) {
        for (; r + kFlight <= r1; r += kFlight) split_rows<DT, true, kFlight>(P, col, n, r, sg, su);
        for (; r < r1; ++r) split_rows<DT, true, 1>(P, col, n, r, sg, su);
    } else if (n > 0) {
        for (; r < r1; ++r) split_rows<DT, false, 1>(P, col, n, r, sg, su);
    }
    if (!P.sums) return;
    float4 s[4] = {make_float4(sg[0], sg[1], sg[2], sg[3]), make_float4(sg[4], sg[5], sg[6], sg[7]), make_float4(su[0], su[1], su[2], su[3]),
                   make_float4(su[4], su[5], su[6], su[7])};
    if (blockDim.y > 1) {
        // the block's workers, in order
#pragma unroll
        for (int j = 0; j < 4; ++j) turned[thread][j] = s[j];
        __syncthreads();
        if (threadIdx.y > 0) return;
        for (int y = 1; y < blockDim.y; ++y)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 v = turned[y * blockDim.x + threadIdx.x][j];
                s[j] = make_float4(s[j].x + v.x, s[j].y + v.y, s[j].z + v.z, s[j].w + v.w);
            }
    }
    if (n == 0) return;
    float4* q = reinterpret_cast<float4*>(P.sums + (int64_t)by * 2 * P.ld + col);
    q[0] = s[0];
    q[1] = s[1];
    q = reinterpret_cast<float4*>(P.sums + ((int64_t)by * 2 + 1) * P.ld + col);
    q[0] = s[2];
    q[1] = s[3];
}

// The tickets alone, where nothing else precedes the products.
__global__ void __launch_bounds__(256) gated_tickets_kernel(uint32_t* tickets, int n)
{
    after_earlier_work();
    for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) tickets[i] = 0;
}

// The biases' gradients where no product is asked for: a warp 32 columns.
template <int DT>
__global__ void __launch_bounds__(128) gated_bias_kernel(const __grid_constant__ GatedParams<kBackward> P)
{
    after_earlier_work();
    const int64_t c0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 5)) * 32;
    if (c0 < P.cols) add_workers<DT>(P.sums + blockIdx.y * P.ld, P.ld, P.workers, c0, P.cols, P.db[blockIdx.y], P.accumulate, threadIdx.x & 31);
}

// ------------------------------------------------------------------ few rows
//
// Up to kFewRows rows of x: reading both weights is all there is.  fp32 products on the plain cores straight from
// the loads, no tiles and one launch, for operands on the 16-byte grid.
constexpr int kFewRows = 2;
constexpr int kFewWarps = 8;                          // warps a block
constexpr int kFewParts = 8;                          // (in, out): blocks a cluster at most
constexpr int kFewResident = 3;                       // (in, out): blocks an SM

struct FewParams {
    const uint16_t *x, *w[2];
    const uint16_t* bias[2];
    uint16_t *h, *gate, *up;
    int64_t ld_x, ld_w[2], ld_h, ld_gate, ld_up;
    int32_t M, N, K;   // K (and N where the weights are stored along it) in eights; rows of x and W start on 16 bytes
    int32_t act, split;   // split: (out, in): warps along K
};

template <int DT>
__device__ __forceinline__ void few_finish(const FewParams& P, int64_t row, int64_t col, float g, float u)
{
    if (P.bias[0]) g += widen1<DT>(P.bias[0][col]);
    if (P.bias[1]) u += widen1<DT>(P.bias[1][col]);
    if (P.gate) P.gate[row * P.ld_gate + col] = narrow1<DT>(g);
    if (P.up) P.up[row * P.ld_up + col] = narrow1<DT>(u);
    P.h[row * P.ld_h + col] = narrow1<DT>(act_value(g, P.act) * u);
}

// Weights stored (out, in): a warp takes a row of each and every `split`-th 256 elements of them.
template <int DT, int ROWS>
__global__ void __launch_bounds__(32 * kFewWarps, 4) gated_few_kernel(const __grid_constant__ FewParams P)
{
    constexpr int U = 2;
    __shared__ float part[kFewWarps][ROWS * 2];
    after_earlier_work();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, ways = P.split, sub = warp % ways;
    const int64_t n = (int64_t)blockIdx.x * (kFewWarps / ways) + warp / ways, nc = min(n, (int64_t)P.N - 1);
    const uint16_t *x[ROWS], *w[2];   // the last row again where there are fewer
#pragma unroll
    for (int m = 0; m < ROWS; ++m) x[m] = P.x + min(m, P.M - 1) * P.ld_x;
#pragma unroll
    for (int c = 0; c < 2; ++c) w[c] = P.w[c] + nc * P.ld_w[c];
    F2 acc[ROWS][2];
#pragma unroll
    for (int m = 0; m < ROWS; ++m)
#pragma unroll
        for (int c = 0; c < 2; ++c) acc[m][c] = both(0.0f);
    const int64_t step = ways * 256;
    int64_t k = sub * 256 + lane * 8;
    for (; k + (U - 1) * step < P.K; k += U * step) few_eights<DT, U, ROWS, 2>(x, w, k, step, acc);
    for (; k < P.K; k += step) few_eights<DT, 1, ROWS, 2>(x, w, k, step, acc);
#pragma unroll
    for (int m = 0; m < ROWS; ++m)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float a, b;
            split(acc[m][c], a, b);
            a += b;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
            if (lane == 0) part[warp][m * 2 + c] = a;
        }
    __syncthreads();
    const int i = threadIdx.x;
    if (i >= kFewWarps / ways * ROWS) return;
    const int g = i / ROWS, m = i % ROWS;
    const int64_t col = (int64_t)blockIdx.x * (kFewWarps / ways) + g;
    if (m >= P.M || col >= P.N) return;
    float a = 0.0f, b = 0.0f;
    for (int v = 0; v < ways; ++v) {
        a += part[g * ways + v][m * 2];
        b += part[g * ways + v][m * 2 + 1];
    }
    few_finish<DT>(P, m, col, a, b);
}

// Weights stored (in, out): a block takes 64 columns of both and one part of K, half of its warps each weight, a
// thread eight columns and eight rows at a time, so that its eight elements of x are one load; the blocks of a
// cluster are the parts, summed in order.
template <int DT, int ROWS>
__global__ void __launch_bounds__(32 * kFewWarps, kFewResident) gated_few_deep_kernel(const __grid_constant__ FewParams P)
{
    constexpr int kDeep = kFewWarps / 2;              // warps along K
    __shared__ float part[kFewWarps][ROWS * 64];
    __shared__ float whole[2 * ROWS * 64];
    after_earlier_work();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, across = (lane & 7) * 8, which = warp / kDeep;
    // past the last column: that column's eight again
    const int64_t ld = P.ld_w[which];
    const uint16_t* w = P.w[which] + min((int64_t)blockIdx.x * 64 + across, (int64_t)P.N - 8);
    const int64_t per = (P.K / 8 + gridDim.y - 1) / gridDim.y * 8, end = min((int64_t)P.K, (blockIdx.y + 1) * per);
    F2 acc[ROWS][4];
#pragma unroll
    for (int m = 0; m < ROWS; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[m][j] = both(0.0f);
    for (int64_t k = blockIdx.y * per + warp % kDeep * 32 + (lane >> 3) * 8; k < end; k += kDeep * 32) {
        uint4 wv[8], xv[ROWS];
#pragma unroll
        for (int u = 0; u < 8; ++u) wv[u] = __ldcs(reinterpret_cast<const uint4*>(w + (k + u) * ld));
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
    float z[2] = {0.0f, 0.0f};
    if (mine) {
#pragma unroll
        for (int v = 0; v < kDeep; ++v) {
            z[0] += part[v][i];
            z[1] += part[kDeep + v][i];
        }
    }
    if (gridDim.y > 1) {
        if (mine) {
            whole[i] = z[0];
            whole[ROWS * 64 + i] = z[1];
        }
        cluster_sync();
        if (mine && blockIdx.y == 0) {
            for (uint32_t r = 1; r < gridDim.y; ++r)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t at;
                    float v;
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(&whole[c * ROWS * 64 + i])), "r"(r));
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
                    z[c] += v;
                }
        }
        cluster_sync();   // a block's shared memory outlives the reads of it
    }
    if (mine && blockIdx.y == 0) few_finish<DT>(P, m, col, z[0], z[1]);
}

// ------------------------------------------------------------------ host

// The shape of the tiles: 256 x 256 on a pair of SMs, an inner block of which takes 0.31 us, or 128 x 128 on one, 0.22 to
// 0.3, the more SMs load the more, whichever is sooner done (with 0.23 gradients of 300 tokens 2000 -> 5000 took 57 us
// instead of 46, of 2500 tokens 768 -> 2048 45 instead of 41).
struct Shape {
    int cg, bn;
    double block_us;
    int workers() const { return kGb300Sms / cg; }
    int64_t rows(int64_t m) const { return div_up(m, kBM * cg); }
    int64_t cols(int64_t n) const { return div_up(n, bn); }
};
constexpr Shape kShapes[] = {{2, 256, 0.31}, {1, 128, 0.25}};

// n1 items of us1 and n2 of us2 dealt so that the worker with most has least; *us: its time.
Deal deal_out(const Shape& S, int64_t n1, double us1, int64_t n2, double us2, double* us)
{
    const int64_t w = std::min<int64_t>(S.workers(), std::max<int64_t>(1, n1 + n2)), q = n1 / w, ahead = n1 % w;
    Deal best{(int32_t)n1, (int32_t)n2, (int32_t)w, (int32_t)ahead, 0, 0};
    if (n2 == 0) {
        *us = (q + (ahead > 0)) * us1;
        return best;
    }
    *us = 1e30;
    // where both kinds of workers would end together, and whole numbers around it
    const int64_t even = std::max<int64_t>(0, (int64_t)(((double)n2 - (double)(w - ahead) * us1 / us2) / (double)w) - 1);
    for (int64_t more = even; more <= even + 3; ++more) {
        const int64_t left = std::max<int64_t>(0, n2 - more * ahead), rest = div_up(left, w - ahead);
        const double most = std::max(ahead > 0 ? (q + 1) * us1 + more * us2 : 0.0, q * us1 + rest * us2);
        if (most >= *us) continue;
        *us = most;
        best.more = (int32_t)more;
        best.rest = (int32_t)rest;
    }
    return best;
}

// How a launch is cut: the tiles' shape, and of either kind how many there are and the parts of their inner dimension.
struct Cut {
    Shape shape = kShapes[0];
    int64_t tiles1 = 0, tiles2 = 0;
    int splits1 = 1, splits2 = 1, per1 = 1, per2 = 1;
    Deal deal{0, 0, 1, 0, 0, 0};
    double us = 1e30;
    int64_t tiles_in_parts() const { return (splits1 > 1 ? tiles1 : 0) + (splits2 > 1 ? tiles2 : 0); }
    int64_t partial_bytes() const { return (splits1 > 1 ? tiles1 * splits1 : 0) * tile_bytes() + (splits2 > 1 ? tiles2 * splits2 : 0) * tile_bytes(); }
    int64_t tile_bytes() const { return 4ll * kBM * shape.cg * shape.bn; }
    int64_t tickets() const { return tiles_in_parts() * kEpiWarps * shape.cg; }
};

// One tile, or one part of `splits`, of kb inner blocks: 256 x 256 cost 3.8 us beside them (128 x 128: 1.5), a part 5 us (2.5)
// more and its share of the sum (with 1.2 for either tile, 300 tokens 2048 -> 2048 took 24.5 us instead of 12.3,
// gradients of 500 tokens 1024 -> 1024 22.8 instead of 16.6).
double tile_us(const Shape& S, int64_t kb, int splits)
{
    return (double)kb * S.block_us + (S.cg == 2 ? 3.8 : 1.5) + (splits > 1 ? (S.cg == 2 ? 5.0 : 2.5) + 0.15 * splits : 0.0);
}

// May n tiles of kb inner blocks be in `ways` parts?  Each has four blocks at least; a worker at most 8 parts of either
// kind of tile, so that the sums take at most 160 MB for each kind: 320 where dx and the weights' gradients are both in parts.
bool divides(const Shape& S, int64_t n, int64_t kb, int ways, int64_t* per)
{
    *per = div_up(std::max<int64_t>(kb, 1), ways);
    return ways == 1 || (n > 0 && *per >= 4 && div_up(kb, *per) == ways && n * ways < 8 * S.workers());
}

// Tiles of two kinds, in parts or whole, and end_us after them, where that is sooner done than *best.
void consider(const Shape& S, int64_t n1, int64_t kb1, int ways1, int64_t n2, int64_t kb2, int ways2, double end_us, Cut* best)
{
    int64_t per1, per2;
    if (!divides(S, n1, kb1, ways1, &per1) || !divides(S, n2, kb2, ways2, &per2)) return;
    double us = 0.0;
    const Deal D = deal_out(S, n1 * ways1, tile_us(S, per1, ways1), n2 * ways2, tile_us(S, per2, ways2), &us);
    us += end_us;
    if (us >= best->us) return;
    best->us = us;
    best->shape = S;
    best->tiles1 = n1;
    best->tiles2 = n2;
    best->splits1 = ways1;
    best->splits2 = ways2;
    best->per1 = (int)per1;
    best->per2 = (int)per2;
    best->deal = D;
}

// Products of m1 x n1 over kb1 inner blocks and `count2` of m2 x n2 over kb2.
Cut choose_cut(int64_t m1, int64_t n1, int64_t kb1, int64_t count2, int64_t m2, int64_t n2, int64_t kb2)
{
    static const int kWays[] = {1, 2, 4, 8, 16, 32};
    Cut best;
    for (const Shape& S : kShapes)
        for (const int ways1 : kWays)
            for (const int ways2 : kWays)
                consider(S, S.rows(m1) * S.cols(n1), kb1, ways1, count2 * S.rows(m2) * S.cols(n2), kb2, ways2, 0.0, &best);
    return best;
}

// One product: whole tiles, and parts of those that would not fill a round (or of all).  The last sums are nothing's to
// hide behind: 0.25 us a part (256 x 256 tiles 0.55) and 0.03 (0.08) for each tile in parts.  16 tokens 4096 -> 11008,
// 172 tiles for 152 workers, 42 -> 37 us; 64 tokens 8192 -> 256, four tiles, 30 -> 13.7.  Less than a hundredth is not
// worth the sums: 8192 tokens 4096 -> 11008, 16 tiles beyond 36 rounds, lose 10 us by them.
Cut choose_cut(int64_t m, int64_t n, int64_t kb)
{
    constexpr int kMostWays = 32;
    Cut best;
    for (const Shape& S : kShapes) {
        const int64_t tiles = S.rows(m) * S.cols(n), over = tiles % S.workers();
        consider(S, tiles, kb, 1, 0, 0, 1, 0.0, &best);
        const double margin = 0.01 * tile_us(S, kb, 1) * (double)div_up(tiles, S.workers());
        for (const int64_t parted : {over, tiles})
            for (int ways = 2; ways <= kMostWays; ++ways)
                consider(S, tiles - parted, kb, 1, parted, kb, ways, margin + ways * (S.cg == 2 ? 0.55 + 0.08 * (double)parted : 0.25 + 0.03 * (double)parted), &best);
    }
    return best;
}

template <int CG, int BN, int MODE, int DT>
zero_status_t launch_gated(const GatedParams<MODE>& P, cudaStream_t s)
{
    using S = GemmShape<CG, BN>;
    const cudaError_t set = allow_shared<gated_kernel<CG, BN, MODE, DT>>(S::kSmem);
    if (set != cudaSuccess) return cuda_fail(set, "zero_gated: shared memory");
    const cudaError_t e = launch_after(gated_kernel<CG, BN, MODE, DT>, CG * P.deal.w, kGemmThreads, S::kSmem, s, P);
    return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "zero_gated: launch");
}

template <int MODE>
zero_status_t launch_gated(const GatedParams<MODE>& P, const Shape& c, bool bf, cudaStream_t s)
{
    if (c.cg == 2) return bf ? launch_gated<2, 256, MODE, ZERO_BF16>(P, s) : launch_gated<2, 256, MODE, ZERO_FP16>(P, s);
    return bf ? launch_gated<1, 128, MODE, ZERO_BF16>(P, s) : launch_gated<1, 128, MODE, ZERO_FP16>(P, s);
}

// fp32 accumulators; operand type; which operands lie along their rows; N / 8; M / 16
uint32_t product_desc(bool bf, bool a_mn, bool b_mn, const Shape& c)
{
    return (1u << 4) | ((bf ? 1u : 0u) << 7) | ((bf ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(c.bn >> 3) << 17) | ((uint32_t)((kBM * c.cg) >> 4) << 24);
}

template <int DT, int ROWS>
zero_status_t launch_few(FewParams P, bool in_out, cudaStream_t s)
{
    cudaError_t e;
    if (!in_out) {
        // warps along K until there are sixteen an SM, by 256 elements in turn; the last shares may be short or empty
        P.split = 1;
        while (P.split < kFewWarps && (int64_t)P.N * P.split < 16 * kGb300Sms && P.split * 256 < P.K) P.split *= 2;
        e = launch_after(gated_few_kernel<DT, ROWS>, (unsigned)div_up(P.N, kFewWarps / P.split), 32 * kFewWarps, 0, s, P);
    } else {
        // as many parts of K as are resident at one time; each has at least 128 rows of the weights
        const int64_t blocks = div_up(P.N, 64);
        int parts = 1;
        while (parts < kFewParts && 2 * parts * blocks <= kFewResident * kGb300Sms && 256 * parts <= P.K) parts *= 2;
        e = launch_clusters_after(gated_few_deep_kernel<DT, ROWS>, dim3(1, parts), dim3((unsigned)blocks, parts), 32 * kFewWarps, 0, s, P);
    }
    return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "zero_gated: launch");
}

template <int DT>
zero_status_t launch_few(const FewParams& P, bool in_out, cudaStream_t s)
{
    return P.M == 1 ? launch_few<DT, 1>(P, in_out, s) : launch_few<DT, 2>(P, in_out, s);
}

// How the pass over dh, g and u is cut: threads across the columns (eight each) and workers a block, rows a worker:
// about six blocks an SM where there are rows for them, and two rows a worker at least.
struct SplitCut {
    int tx = 256, ty = 1, chunk = 1;
    int64_t workers = 0;
    int64_t groups() const { return div_up(workers, ty); }   // blocks across the rows, each of which writes its sums
};

SplitCut split_cut(int64_t rows, int64_t cols)
{
    SplitCut c;
    while (c.tx > 32 && (int64_t)c.tx * 4 >= cols) c.tx /= 2;
    c.ty = 256 / c.tx;
    const int64_t across = std::max<int64_t>(1, div_up(cols, (int64_t)c.tx * 8));
    const int64_t want = std::max<int64_t>(1, 6 * kGb300Sms * c.ty / across);
    c.chunk = (int)std::max<int64_t>(2, div_up(std::max<int64_t>(rows, 1), want));
    c.workers = div_up(rows, c.chunk);
    return c;
}

constexpr int64_t kMaxSize = ZERO_LINEAR_MAX_SIZE;   // tile coordinates stay 32-bit
constexpr int64_t kMaxElements = (int64_t)1 << 42;   // so do counts of tiles

// Everything a call needs, checked: strides filled in, and where its pieces lie in the workspace.
struct Gated {
    zero_gated_t a;
    bool bf = true, few = false, copy[3] = {false, false, false};   // x, Wg, Wu
    int64_t w_rows = 0, w_cols = 0;        // as stored
    int64_t ld8[3] = {0, 0, 0}, at_copy[3] = {0, 0, 0};
    int64_t ld_d = 0, at_dg = 0, at_du = 0, at_sums = 0, bytes = 0;
    int64_t at_partial = 0, at_tickets = 0;
    bool make_d = false, make_sums = false;
    SplitCut cut;
    Cut tiles;
};

zero_status_t lay_out(const zero_gated_t* in, bool back, Gated* L, const char* who)
{
    const std::string w = std::string(who) + ": ";
    if (!in) return fail(ZERO_EINVAL, w + "NULL arguments");
    L->a = *in;
    zero_gated_t& a = L->a;
    if (a.rows < 0 || a.in_features < 0 || a.out_features < 0) return fail(ZERO_EINVAL, w + "negative size");
    if (a.rows > kMaxSize || a.in_features > kMaxSize || a.out_features > kMaxSize)
        return fail(ZERO_ERANGE, w + "a size beyond ZERO_LINEAR_MAX_SIZE");
    for (const int64_t n : {a.rows * a.in_features, a.rows * a.out_features, a.in_features * a.out_features})
        if (n > kMaxElements) return fail(ZERO_ERANGE, w + "a matrix beyond 2^42 elements");
    if (a.dtype16 != ZERO_BF16 && a.dtype16 != ZERO_FP16) return fail(ZERO_EINVAL, w + "bad dtype16");
    if (a.layout != ZERO_WEIGHT_OUT_IN && a.layout != ZERO_WEIGHT_IN_OUT) return fail(ZERO_EINVAL, w + "bad layout");
    if (a.activation < ZERO_ACT_NONE || a.activation > ZERO_ACT_SILU) return fail(ZERO_EINVAL, w + "bad activation");
    if (a.flags & ~(back ? ZERO_GATED_ACCUMULATE : 0)) return fail(ZERO_EINVAL, w + "unknown flag");
    L->bf = a.dtype16 == ZERO_BF16;
    const bool out_in = a.layout == ZERO_WEIGHT_OUT_IN;
    L->w_rows = out_in ? a.out_features : a.in_features;
    L->w_cols = out_in ? a.in_features : a.out_features;
    struct {
        int64_t* ld;
        int64_t cols;
    } strides[] = {{&a.ld_x, a.in_features},   {&a.ld_w_gate, L->w_cols}, {&a.ld_w_up, L->w_cols},   {&a.ld_h, a.out_features}, {&a.ld_gate, a.out_features},
                   {&a.ld_up, a.out_features}, {&a.ld_dh, a.out_features}, {&a.ld_dx, a.in_features}, {&a.ld_dw_gate, L->w_cols}, {&a.ld_dw_up, L->w_cols}};
    for (auto& s : strides) {
        if (*s.ld == 0) *s.ld = s.cols;
        if (*s.ld < s.cols) return fail(ZERO_EINVAL, w + "a row stride is shorter than its row");
        if (*s.ld > ((int64_t)1 << 38)) return fail(ZERO_ERANGE, w + "a row stride beyond 2^38");
    }
    const void* every[] = {a.x, a.w_gate, a.w_up, a.b_gate, a.b_up, a.h, a.gate, a.up, a.dh, a.dx, a.dw_gate, a.dw_up, a.db_gate, a.db_up};
    for (const void* p : every)
        if (!aligned(p, 2)) return fail(ZERO_EALIGN, w + "a pointer is not aligned to 2 bytes");
    const bool any_out = a.rows > 0 && a.out_features > 0, any_in = any_out && a.in_features > 0;
    if (!back) {
        if (any_out && !a.h) return fail(ZERO_EINVAL, w + "h is NULL");
        if (any_in && (!a.x || !a.w_gate || !a.w_up)) return fail(ZERO_EINVAL, w + "x, w_gate or w_up is NULL");
        if (any_out && ((a.gate && (a.gate == a.h || a.gate == a.up)) || (a.up && a.up == a.h)))
            return fail(ZERO_EINVAL, w + "two outputs are one buffer");
    } else {
        if (!a.dx && !a.dw_gate && !a.dw_up && !a.db_gate && !a.db_up) return fail(ZERO_EINVAL, w + "no gradient asked for");
        if (any_out && (!a.dh || !a.gate || !a.up)) return fail(ZERO_EINVAL, w + "dh, gate or up is NULL");
        if (any_in && ((a.dx && (!a.w_gate || !a.w_up)) || ((a.dw_gate || a.dw_up) && !a.x)))
            return fail(ZERO_EINVAL, w + "x, w_gate or w_up is NULL");
        if ((a.dw_gate && a.dw_gate == a.dw_up) || (a.db_gate && a.db_gate == a.db_up))
            return fail(ZERO_EINVAL, w + "two gradients are one buffer");
    }
    // the pieces of the workspace
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += up(bytes, 256);
        return here;
    };
    const void* source[3] = {a.x, a.w_gate, a.w_up};
    const int64_t ld[3] = {a.ld_x, a.ld_w_gate, a.ld_w_up};
    const int64_t rows[3] = {a.rows, L->w_rows, L->w_rows}, cols[3] = {a.in_features, L->w_cols, L->w_cols};
    const bool weights = !back || a.dx, input = !back || a.dw_gate || a.dw_up;
    const bool use[3] = {input, weights, weights};
    bool ready = true;
    for (int i = 0; i < 3; ++i) ready = ready && tma_ready(source[i], ld[i]);
    L->few = !back && any_in && a.rows <= kFewRows && a.in_features % 8 == 0 && ready && (out_in || a.out_features % 8 == 0);
    for (int i = 0; i < 3; ++i) {
        L->ld8[i] = ld[i];
        L->copy[i] = any_in && use[i] && !L->few && !tma_ready(source[i], ld[i]);
        if (L->copy[i]) {
            L->ld8[i] = up(cols[i], 8);
            L->at_copy[i] = take(2 * rows[i] * L->ld8[i]);
        }
    }
    if (back && any_out) {
        L->make_d = any_in && (a.dx || a.dw_gate || a.dw_up);
        L->make_sums = a.db_gate || a.db_up;
        L->ld_d = up(a.out_features, 8);
        L->cut = split_cut(a.rows, a.out_features);
        if (L->make_d) {
            L->at_dg = take(2 * a.rows * L->ld_d);
            L->at_du = take(2 * a.rows * L->ld_d);
        }
        if (L->make_sums) L->at_sums = take(8 * L->cut.groups() * L->ld_d);
    }
    if (any_in && !L->few && (!back || L->make_d)) {
        const int weights = (a.dw_gate != nullptr) + (a.dw_up != nullptr);
        const int64_t kb_k = div_up(a.in_features, kBK), kb_n = div_up(a.out_features, kBK), kb_m = div_up(a.rows, kBK);
        L->tiles = back ? choose_cut(a.dx ? a.rows : 0, a.in_features, 2 * kb_n, weights, L->w_rows, L->w_cols, kb_m)
                        : choose_cut(a.rows, 2 * a.out_features, kb_k);
        if (L->tiles.partial_bytes() > 0) {
            L->at_partial = take(L->tiles.partial_bytes());
            L->at_tickets = take(4 * L->tiles.tickets());
        }
    }
    L->bytes = at;
    return ZERO_OK;
}

zero_status_t check_workspace(const Gated& L, const void* workspace, int64_t bytes, const char* who)
{
    if (L.bytes == 0) return ZERO_OK;
    if (!workspace) return fail(ZERO_EINVAL, std::string(who) + ": workspace is NULL");
    if (!aligned(workspace, 16)) return fail(ZERO_EALIGN, std::string(who) + ": workspace not 16-byte aligned");
    if (bytes < L.bytes)
        return fail(ZERO_ERANGE, std::string(who) + ": workspace of " + std::to_string(bytes) + " bytes, " + std::to_string(L.bytes) + " needed");
    return ZERO_OK;
}

// The copies that the call needs, and its tickets, into S; the operands become theirs.
void plan_copies(const Gated& L, char* ws, const void* (&operand)[3], SplitParams* S)
{
    const zero_gated_t& a = L.a;
    std::memset(S, 0, sizeof(*S));
    S->tickets = reinterpret_cast<uint32_t*>(ws + L.at_tickets);
    S->n_tickets = (int32_t)L.tiles.tickets();
    const int64_t ld[3] = {a.ld_x, a.ld_w_gate, a.ld_w_up};
    const void* source[3] = {a.x, a.w_gate, a.w_up};
    for (int i = 0; i < 3; ++i) {
        operand[i] = source[i];
        if (!L.copy[i]) continue;
        AlignJob& J = S->copy[i];
        J.src = static_cast<const uint16_t*>(source[i]);
        J.dst = reinterpret_cast<uint16_t*>(ws + L.at_copy[i]);
        J.ld_src = ld[i];
        J.ld = L.ld8[i];
        J.rows = i == 0 ? a.rows : L.w_rows;
        J.cols = i == 0 ? a.in_features : L.w_cols;
        S->copy_blocks[i] = grid_of(div_up(J.rows * div_up(J.cols, 8), kCopies), kGb300Sms, 8);
        operand[i] = J.dst;
    }
}

zero_status_t launch_split(const Gated& L, const SplitParams& S, cudaStream_t s)
{
    const int64_t blocks = (int64_t)S.blocks + S.copy_blocks[0] + S.copy_blocks[1] + S.copy_blocks[2];
    cudaError_t e = cudaSuccess;
    if (blocks == 0) {
        if (S.n_tickets > 0) e = launch_after(gated_tickets_kernel, grid_of(S.n_tickets, kGb300Sms, 1), 256, 0, s, S.tickets, (int)S.n_tickets);
        return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "zero_gated: launch");
    }
    const dim3 threads(L.cut.tx, L.cut.ty);
    e = L.bf ? launch_after(split_kernel<ZERO_BF16>, (unsigned)blocks, threads, 0, s, S)
             : launch_after(split_kernel<ZERO_FP16>, (unsigned)blocks, threads, 0, s, S);
    return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "zero_gated: launch");
}

Matrix16 matrix(void* p, int64_t ld, int64_t rows, int64_t cols)
{
    return Matrix16{static_cast<uint16_t*>(p), ld, rows, cols, vec_flag(p, ld, 1)};
}

// The product's parts, after *tiles tiles and *parts parts of others.
void set_parts(Product* Q, int splits, int per, int64_t* tiles, int64_t* parts)
{
    Q->splits = splits;
    Q->k_per_split = per;
    Q->tile0 = (int32_t)*tiles;
    Q->part0 = (int32_t)*parts;
    if (splits == 1) return;
    *tiles += (int64_t)Q->tiles_m * Q->tiles_n;
    *parts += (int64_t)Q->tiles_m * Q->tiles_n * splits;
}

// Zeros for a gradient that sums over nothing.
cudaError_t zeros(void* p, int64_t ld, int64_t rows, int64_t cols, cudaStream_t s)
{
    return p && rows > 0 && cols > 0 ? cudaMemset2DAsync(p, (size_t)ld * 2, 0, (size_t)cols * 2, (size_t)rows, s) : cudaSuccess;
}

}  // namespace

cudaError_t take_gated_error(uint32_t* word, void* stream) { return take_error_word(g_gated_error, word, static_cast<cudaStream_t>(stream)); }

}  // namespace zero

using namespace zero;

extern "C" {

zero_status_t zero_gated_workspace(const zero_gated_t* a, int backward, int64_t* bytes)
try {
    if (!bytes) return fail(ZERO_EINVAL, "zero_gated_workspace: NULL argument");
    Gated L;
    const zero_status_t st = lay_out(a, backward != 0, &L, "zero_gated_workspace");
    if (st == ZERO_OK) *bytes = L.bytes;
    return st;
}
catch (...) {
    return exception_status("zero_gated_workspace");
}

zero_status_t zero_gated(const zero_gated_t* args, void* workspace, int64_t workspace_bytes, void* stream)
try {
    Gated L;
    zero_status_t st = lay_out(args, false, &L, "zero_gated");
    if (st == ZERO_OK) st = check_workspace(L, workspace, workspace_bytes, "zero_gated");
    if (st != ZERO_OK) return st;
    const zero_gated_t& a = L.a;
    if (a.rows == 0 || a.out_features == 0) return ZERO_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool in_out = a.layout == ZERO_WEIGHT_IN_OUT;
    if (L.few) {
        FewParams P;
        std::memset(&P, 0, sizeof(P));
        P.x = static_cast<const uint16_t*>(a.x);
        P.w[0] = static_cast<const uint16_t*>(a.w_gate);
        P.w[1] = static_cast<const uint16_t*>(a.w_up);
        P.bias[0] = static_cast<const uint16_t*>(a.b_gate);
        P.bias[1] = static_cast<const uint16_t*>(a.b_up);
        P.h = static_cast<uint16_t*>(a.h);
        P.gate = static_cast<uint16_t*>(a.gate);
        P.up = static_cast<uint16_t*>(a.up);
        P.ld_x = a.ld_x;
        P.ld_w[0] = a.ld_w_gate;
        P.ld_w[1] = a.ld_w_up;
        P.ld_h = a.ld_h;
        P.ld_gate = a.ld_gate;
        P.ld_up = a.ld_up;
        P.M = (int32_t)a.rows;
        P.N = (int32_t)a.out_features;
        P.K = (int32_t)a.in_features;
        P.act = a.activation;
        return L.bf ? launch_few<ZERO_BF16>(P, in_out, s) : launch_few<ZERO_FP16>(P, in_out, s);
    }
    GatedParams<kForward> P;
    std::memset(&P, 0, sizeof(P));
    P.out[0] = matrix(a.h, a.ld_h, a.rows, a.out_features);
    P.out[1] = matrix(a.gate, a.ld_gate, a.rows, a.out_features);
    P.out[2] = matrix(a.up, a.ld_up, a.rows, a.out_features);
    P.bias[0] = static_cast<const uint16_t*>(a.b_gate);
    P.bias[1] = static_cast<const uint16_t*>(a.b_up);
    P.bias_vec = vec_flag(a.b_gate, 0, 1) | vec_flag(a.b_up, 0, 2);
    P.act = a.activation;
    if (a.in_features == 0) {
        const int grid = grid_of(a.rows * a.out_features, kGb300Sms, 8);
        const cudaError_t e = L.bf ? launch_after(gated_empty_kernel<ZERO_BF16>, grid, 256, 0, s, P) : launch_after(gated_empty_kernel<ZERO_FP16>, grid, 256, 0, s, P);
        return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "zero_gated: launch");
    }
    char* ws = static_cast<char*>(workspace);
    const void* operand[3];
    SplitParams S;
    plan_copies(L, ws, operand, &S);
    st = launch_split(L, S, s);
    if (st != ZERO_OK) return st;
    const Shape c = L.tiles.shape;
    Product& Q = P.part[0];
    // few rows: no zeros are copied for the rest, whose results are not stored
    P.a_rows = c.cg == 1 && a.rows < kBM ? (int32_t)up(a.rows, 8) : kBM;
    st = encode(&Q.a[0], Operand{operand[0], a.rows, a.in_features, L.ld8[0], false}, a.dtype16, P.a_rows, "zero_gated");
    for (int i = 0; i < 2 && st == ZERO_OK; ++i)
        st = encode(&Q.b[i], Operand{operand[1 + i], a.out_features, a.in_features, L.ld8[1 + i], in_out}, a.dtype16, c.cg == 2 ? kBM : kBM / 2, "zero_gated");
    if (st != ZERO_OK) return st;
    Q.tiles_m = (int32_t)c.rows(a.rows);
    Q.tiles_n = (int32_t)div_up(a.out_features, c.bn / 2);
    Q.k_blocks = (int32_t)div_up(a.in_features, kBK);
    Q.b_mn = in_out;
    Q.idesc = product_desc(L.bf, false, in_out, c);
    Q.splits = L.tiles.splits2;
    Q.k_per_split = L.tiles.per2;
    P.deal = L.tiles.deal;
    P.partial = reinterpret_cast<float4*>(ws + L.at_partial);
    P.tickets = reinterpret_cast<uint32_t*>(ws + L.at_tickets);
    return launch_gated<kForward>(P, c, L.bf, s);
}
catch (...) {
    return exception_status("zero_gated");
}

zero_status_t zero_gated_backward(const zero_gated_t* args, void* workspace, int64_t workspace_bytes, void* stream)
try {
    Gated L;
    zero_status_t st = lay_out(args, true, &L, "zero_gated_backward");
    if (st == ZERO_OK) st = check_workspace(L, workspace, workspace_bytes, "zero_gated_backward");
    if (st != ZERO_OK) return st;
    const zero_gated_t& a = L.a;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    const bool accumulate = a.flags & ZERO_GATED_ACCUMULATE, out_in = a.layout == ZERO_WEIGHT_OUT_IN;
    const int64_t m = a.rows, k = a.in_features, n = a.out_features;
    if (m == 0 || n == 0) {
        // sums over nothing
        cudaError_t e = zeros(a.dx, a.ld_dx, m, k, s);
        if (!accumulate) {
            if (e == cudaSuccess) e = zeros(a.dw_gate, a.ld_dw_gate, L.w_rows, L.w_cols, s);
            if (e == cudaSuccess) e = zeros(a.dw_up, a.ld_dw_up, L.w_rows, L.w_cols, s);
            if (e == cudaSuccess) e = zeros(a.db_gate, n, 1, n, s);
            if (e == cudaSuccess) e = zeros(a.db_up, n, 1, n, s);
        }
        return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "zero_gated_backward: memset");
    }
    const void* operand[3];
    SplitParams S;
    plan_copies(L, ws, operand, &S);
    float* sums = L.make_sums ? reinterpret_cast<float*>(ws + L.at_sums) : nullptr;
    if (L.make_d || L.make_sums) {
        S.dh = static_cast<const uint16_t*>(a.dh);
        S.gate = static_cast<const uint16_t*>(a.gate);
        S.up = static_cast<const uint16_t*>(a.up);
        S.dg = L.make_d ? reinterpret_cast<uint16_t*>(ws + L.at_dg) : nullptr;
        S.du = L.make_d ? reinterpret_cast<uint16_t*>(ws + L.at_du) : nullptr;
        S.sums = sums;
        S.rows = m;
        S.cols = n;
        S.ld_dh = a.ld_dh;
        S.ld_gate = a.ld_gate;
        S.ld_up = a.ld_up;
        S.ld = L.ld_d;
        S.act = a.activation;
        S.vec = vec_flag(a.dh, a.ld_dh, 1) && vec_flag(a.gate, a.ld_gate, 1) && vec_flag(a.up, a.ld_up, 1);
        S.chunk = L.cut.chunk;
        S.across = (int32_t)div_up(n, (int64_t)L.cut.tx * 8);
        S.blocks = (int32_t)(S.across * L.cut.groups());
    }
    st = launch_split(L, S, s);
    if (st != ZERO_OK) return st;
    GatedParams<kBackward> P;
    std::memset(&P, 0, sizeof(P));
    P.accumulate = accumulate;
    if (L.make_sums) {
        P.sums = sums;
        P.db[0] = static_cast<uint16_t*>(a.db_gate);
        P.db[1] = static_cast<uint16_t*>(a.db_up);
        P.ld = L.ld_d;
        P.workers = L.cut.groups();
        P.cols = n;
    }
    if (!L.make_d) {
        if (!L.make_sums) return ZERO_OK;
        const dim3 grid((unsigned)div_up(n, 128), 2);
        const cudaError_t e = L.bf ? launch_after(gated_bias_kernel<ZERO_BF16>, grid, 128, 0, s, P) : launch_after(gated_bias_kernel<ZERO_FP16>, grid, 128, 0, s, P);
        return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "zero_gated_backward: launch");
    }
    // dx, then the weights' gradients that are asked for
    const int64_t kb_n = div_up(n, kBK), kb_m = div_up(m, kBK);
    const Cut& T = L.tiles;
    const Shape c = T.shape;
    P.deal = T.deal;
    P.partial = reinterpret_cast<float4*>(ws + L.at_partial);
    P.tickets = reinterpret_cast<uint32_t*>(ws + L.at_tickets);
    int64_t tiles = 0, parts = 0;
    P.a_rows = c.cg == 1 && m < kBM ? (int32_t)up(m, 8) : kBM;
    const Operand d[2] = {{ws + L.at_dg, m, n, L.ld_d, false}, {ws + L.at_du, m, n, L.ld_d, false}};
    int part = 0;
    if (a.dx) {
        Product& Q = P.part[part++];
        Q.out = matrix(a.dx, a.ld_dx, m, k);
        for (int i = 0; i < 2 && st == ZERO_OK; ++i) {
            st = encode(&Q.a[i], d[i], a.dtype16, P.a_rows, "zero_gated_backward");
            if (st == ZERO_OK) st = encode(&Q.b[i], Operand{operand[1 + i], k, n, L.ld8[1 + i], out_in}, a.dtype16, c.bn / c.cg, "zero_gated_backward");
        }
        Q.tiles_m = (int32_t)c.rows(m);
        Q.tiles_n = (int32_t)c.cols(k);
        Q.k_first = (int32_t)kb_n;
        Q.k_blocks = 2 * Q.k_first;
        Q.b_mn = out_in;
        Q.idesc = product_desc(L.bf, false, out_in, c);
        set_parts(&Q, T.splits1, T.per1, &tiles, &parts);
    }
    P.parts_at = part;
    const Operand x{operand[0], k, m, L.ld8[0], true};
    for (int which = 0; which < 2 && st == ZERO_OK; ++which) {
        void* dw = which ? a.dw_up : a.dw_gate;
        if (!dw) continue;
        Product& Q = P.part[part++];
        const Operand z{d[which].p, n, m, L.ld_d, true};
        Q.out = matrix(dw, which ? a.ld_dw_up : a.ld_dw_gate, L.w_rows, L.w_cols);
        st = encode(&Q.a[0], out_in ? z : x, a.dtype16, kBM, "zero_gated_backward");
        if (st == ZERO_OK) st = encode(&Q.b[0], out_in ? x : z, a.dtype16, kBM, "zero_gated_backward");
        Q.tiles_m = (int32_t)c.rows(L.w_rows);
        Q.tiles_n = (int32_t)c.cols(L.w_cols);
        Q.k_blocks = Q.k_first = (int32_t)kb_m;
        Q.a_mn = Q.b_mn = 1;
        Q.idesc = product_desc(L.bf, true, true, c);
        set_parts(&Q, T.splits2, T.per2, &tiles, &parts);
    }
    if (st == ZERO_OK) st = launch_gated<kBackward>(P, c, L.bf, s);
    return st;
}
catch (...) {
    return exception_status("zero_gated_backward");
}

}  // extern "C"
