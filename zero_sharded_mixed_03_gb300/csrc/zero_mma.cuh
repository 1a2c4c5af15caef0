// zero_mma.cuh -- what the translation units with matrix products share: activations, sixteen bytes of a row,
// the fifth-generation tensor cores' copies, products and descriptors, tiles, copies onto the 16-byte grid, and
// tensor maps.
#pragma once

#include <algorithm>
#include <string>

#include <cuda.h>

#include "zero_device.cuh"

namespace zero {
namespace {

constexpr int kBM = 128;                 // rows of a block's tile (a pair of blocks: 256)
constexpr int kBK = 64;                  // inner elements a stage: 128 bytes, one swizzle row
constexpr int kEpiWarps = 8;
constexpr int kGemmThreads = 32 * (4 + kEpiWarps);   // TMA, MMA, TMEM allocation, idle; epilogue
constexpr uint64_t kGemmWaitNs = 2000000000ull;
constexpr int kEpiCols = 32;             // columns an epilogue warp takes at a time
constexpr int kEpiBytes = 32 * kEpiCols * 4;

// ------------------------------------------------------------------ activations

// The logistic function, accurate relative to its value in both tails, down to 2^-126 (z = -87.3): below it is
// 0, as the reciprocal's subnormal results are.  z times it is then off by 2^-119 at most.  One exponential and one
// reciprocal, each an instruction; the plain forms' care for subnormal values costs twice as many.
__device__ __forceinline__ float logistic(float z)
{
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

// The tanh form of gelu is z logistic(2 u), u = sqrt(2 / pi) (z + 0.044715 z^3), and gelu itself
// z erfc(-z / sqrt 2) / 2: neither loses the left tail as 1 + tanh and 1 + erf do.
__device__ __forceinline__ float gelu_arg(float z) { return 1.5957691216057308f * z * (1.0f + 0.044715f * z * z); }

__device__ __forceinline__ float act_value(float z, int act)
{
    switch (act) {
    case ZERO_ACT_RELU: return z > 0.0f ? z : (z <= 0.0f ? 0.0f : z);   // not a number stays so
    case ZERO_ACT_GELU_TANH: return z * logistic(gelu_arg(z));
    case ZERO_ACT_GELU: return 0.5f * z * erfcf(z * -0.7071067811865476f);
    case ZERO_ACT_SILU: return z * logistic(z);
    default: return z;
    }
}

__device__ __forceinline__ float act_slope(float z, int act)
{
    switch (act) {
    case ZERO_ACT_RELU: return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
    case ZERO_ACT_GELU_TANH: {
        // s (1 - s) first: it is 0 where the polynomial leaves fp32's range, and the square stays in it, so that
        // finite numbers have finite slopes (in bf16 |z| goes to 3e38)
        const float s = logistic(gelu_arg(z));
        return s + s * (1.0f - s) * z * (1.5957691216057308f * (1.0f + 0.134145f * fminf(z * z, 1e30f)));
    }
    case ZERO_ACT_GELU:
        return 0.5f * erfcf(z * -0.7071067811865476f) + z * __expf(-0.5f * z * z) * 0.3989422804014327f;
    case ZERO_ACT_SILU: {
        const float s = logistic(z);
        return s * (1.0f + z * (1.0f - s));
    }
    default: return 1.0f;
    }
}

// Eight at a time: one branch for all.
__device__ __forceinline__ void act_values(float (&z)[8], int act)
{
#define ZERO_EACH(A) case A: _Pragma("unroll") for (int j = 0; j < 8; ++j) z[j] = act_value(z[j], A); break
    switch (act) {
        ZERO_EACH(ZERO_ACT_RELU);
        ZERO_EACH(ZERO_ACT_GELU_TANH);
        ZERO_EACH(ZERO_ACT_GELU);
        ZERO_EACH(ZERO_ACT_SILU);
    }
#undef ZERO_EACH
}

__device__ __forceinline__ void act_slopes(float (&z)[8], int act)
{
#define ZERO_EACH(A) case A: _Pragma("unroll") for (int j = 0; j < 8; ++j) z[j] = act_slope(z[j], A); break
    switch (act) {
        ZERO_EACH(ZERO_ACT_RELU);
        ZERO_EACH(ZERO_ACT_GELU_TANH);
        ZERO_EACH(ZERO_ACT_GELU);
        ZERO_EACH(ZERO_ACT_SILU);
    }
#undef ZERO_EACH
}

// ------------------------------------------------------------------ eight columns of one row

template <int DT>
__device__ __forceinline__ void load8(const uint16_t* p, bool vec, int n, float (&x)[8])
{
    if (vec && n == 8) {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        widen2<DT>(w.x, x[0], x[1]);
        widen2<DT>(w.y, x[2], x[3]);
        widen2<DT>(w.z, x[4], x[5]);
        widen2<DT>(w.w, x[6], x[7]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = j < n ? widen1<DT>(p[j]) : 0.0f;
    }
}

template <int DT>
__device__ __forceinline__ void store8(uint16_t* p, bool vec, int n, const float (&x)[8])
{
    if (vec && n == 8) {
        *reinterpret_cast<uint4*>(p) = make_uint4(narrow2<DT>(x[0], x[1]), narrow2<DT>(x[2], x[3]),
                                                  narrow2<DT>(x[4], x[5]), narrow2<DT>(x[6], x[7]));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) p[j] = narrow1<DT>(x[j]);
    }
}

// ------------------------------------------------------------------ tensor-core building blocks

template <int CG>
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    if constexpr (CG == 2)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
            " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar)
            : "memory");
}

template <int CG>
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    if constexpr (CG == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
            "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
            "r"(accumulate)
            : "memory");
}

// Arrive on `bar` (of both blocks of a pair) once every product issued so far is done.
template <int CG>
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    if constexpr (CG == 2)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"((uint16_t)3)
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ uint32_t leader_address(uint32_t addr)   // the pair's first block's copy of `addr`
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}

__device__ __forceinline__ void arrive_cluster(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// 32 lanes x 32 columns of fp32 from TMEM: this thread's lane's columns.
__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&x)[32])
{
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(r[i]);
}

// Shared-memory descriptor of a 128-byte swizzled operand tile.
//   stored along K:  rows of 128 bytes, eight of them an atom of 1 KB; atoms 1 KB apart (stride)
//   stored along MN: 64 elements of MN in 128 bytes, eight K rows an atom; K groups 1 KB apart
//                    (stride), the next 64 of MN one box of kBK rows on (leading: 8 KB)
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, bool mn)
{
    const uint64_t leading = mn ? (kBK * 128) >> 4 : 1, stride = 1024 >> 4;
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (leading << 16) | (stride << 32) | (1ull << 46) | (2ull << 61);
}

// Tile (m, n) of item `t`: groups of 8 tile rows are walked column by column, so that what runs
// at one time shares its operands in L2.
__device__ __forceinline__ void tile_at(int tiles_m, int tiles_n, int t, int& m, int& n)
{
    constexpr int kGroup = 8;
    const int per_group = kGroup * tiles_n, g = t / per_group, in = t - g * per_group;
    const int rows = min(kGroup, tiles_m - g * kGroup);
    n = in / rows;
    m = g * kGroup + (in - n * rows);
}

template <int CG, int BN>
struct GemmShape {
    static constexpr int kBRows = BN / CG;                       // B rows one block stages
    static constexpr int kABytes = kBM * kBK * 2, kBBytes = kBRows * kBK * 2;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kStages = BN == 64 ? 8 : 6;
    static constexpr int kTmemCols = 2 * BN;                     // two accumulators
    static constexpr int kSmem = 1024 + kStages * kStageBytes + kEpiWarps * kEpiBytes + 256;
};

// One lane of a whole warp, in a form that the compiler knows to be one: copies and products are then issued from
// uniform registers.  Behind `lane == 0` it has to expect several, and two copies cost 470 cycles, more than the
// products of an inner block take (128 x 128 tiles).
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// ------------------------------------------------------------------ tiles of 16 bits

// A 16-bit matrix that tiles are read from or written to.
struct Matrix16 {
    uint16_t* p;
    int64_t ld, rows, cols;
    int32_t vec;             // rows start on 16 bytes
};

// Where a warp keeps a 32 x 32 tile of 16 bits: rows of 64 bytes, their 16-byte pieces exchanged so that neither
// eight rows' same pieces nor two rows' four conflict.
constexpr int kTile16Bytes = 32 * 64;

__device__ __forceinline__ uint32_t tile16_at(uint32_t stage, int row, int piece) { return stage + row * 64 + ((piece ^ ((row >> 1) & 3)) << 4); }

// The tile in shared memory to global memory; what is past the matrix is left out.  WHOLE: with a way for tiles that are
// all inside (loads, then stores, and no branch between them), for kernels that little else bounds: more instructions.
template <bool WHOLE>
__device__ __forceinline__ void store_tile16(uint32_t stage, int lane, const Matrix16& D, int64_t row0, int64_t col0)
{
    if (WHOLE && D.vec && row0 + 32 <= D.rows && col0 + 32 <= D.cols) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w) : "r"(tile16_at(stage, i * 8 + (lane >> 2), lane & 3)) : "memory");
        uint16_t* q = D.p + (row0 + (lane >> 2)) * D.ld + col0 + (lane & 3) * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i, q += 8 * D.ld) *reinterpret_cast<uint4*>(q) = v[i];
    } else if (D.vec) {
        const int64_t col = col0 + (lane & 3) * 8;
        const int n = (int)max((int64_t)0, min((int64_t)8, D.cols - col));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + (lane >> 2);
            uint32_t w[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(tile16_at(stage, r, lane & 3)) : "memory");
            if (row0 + r >= D.rows || n == 0) continue;
            uint16_t* q = D.p + (row0 + r) * D.ld + col;
            if (n == 8) {
                *reinterpret_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < n) q[j] = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
            }
        }
    } else if (col0 + lane < D.cols) {
        // a column a lane, so that a warp writes neighbours
        const int rows = (int)min((int64_t)32, D.rows - row0);
#pragma unroll 8
        for (int r = 0; r < rows; ++r) {
            uint16_t v;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(tile16_at(stage, r, lane >> 3) + (lane & 7) * 2) : "memory");
            D.p[(row0 + r) * D.ld + col0 + lane] = v;
        }
    }
}

// The tile of global memory into shared memory; zeros past the matrix.
__device__ __forceinline__ void load_tile16(uint32_t stage, int lane, const Matrix16& D, int64_t row0, int64_t col0)
{
    if (D.vec) {
        const int64_t col = col0 + (lane & 3) * 8;
        const int n = (int)max((int64_t)0, min((int64_t)8, D.cols - col));
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = row0 + i * 8 + (lane >> 2);
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (row >= D.rows || n == 0) continue;
            const uint16_t* q = D.p + row * D.ld + col;
            if (n == 8) {
                v[i] = *reinterpret_cast<const uint4*>(q);
            } else {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = (2 * j < n ? q[2 * j] : 0u) | ((2 * j + 1 < n ? (uint32_t)q[2 * j + 1] : 0u) << 16);
                v[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(tile16_at(stage, i * 8 + (lane >> 2), lane & 3)), "r"(v[i].x), "r"(v[i].y), "r"(v[i].z), "r"(v[i].w) : "memory");
    } else {
#pragma unroll 8
        for (int r = 0; r < 32; ++r) {
            const uint16_t v = row0 + r < D.rows && col0 + lane < D.cols ? D.p[(row0 + r) * D.ld + col0 + lane] : (uint16_t)0;
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(tile16_at(stage, r, lane >> 3) + (lane & 7) * 2), "h"(v) : "memory");
        }
    }
}

// x: row `lane` of the tile in shared memory, rounded once.
template <int DT>
__device__ __forceinline__ void write_tile16(uint32_t stage, int lane, const float (&x)[32])
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(tile16_at(stage, lane, i)), "r"(narrow2<DT>(x[8 * i], x[8 * i + 1])),
                     "r"(narrow2<DT>(x[8 * i + 2], x[8 * i + 3])), "r"(narrow2<DT>(x[8 * i + 4], x[8 * i + 5])),
                     "r"(narrow2<DT>(x[8 * i + 6], x[8 * i + 7]))
                     : "memory");
}

// The same tile at (row0, col0) of a matrix, through shared memory, so that a store instruction writes whole sectors.
template <int DT, bool WHOLE = false>
__device__ __forceinline__ void put_tile(uint32_t stage, int lane, const float (&x)[32], const Matrix16& D, int64_t row0, int64_t col0)
{
    write_tile16<DT>(stage, lane, x);
    __syncwarp();
    store_tile16<WHOLE>(stage, lane, D, row0, col0);
    __syncwarp();
}

// The tile in shared memory (tile16_at's exchange is the 64-byte swizzle; 512-byte aligned) to a tensor map's matrix,
// by a copy that one lane, always the same, starts and that belongs to its bulk group; what is past the matrix is left
// out.
__device__ __forceinline__ void send_tile16(uint32_t stage, const CUtensorMap* map, int64_t row0, int64_t col0)
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (elect_one())
        asm volatile(
            "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n\t"
            "cp.async.bulk.commit_group;" ::"l"(map), "r"((int)col0), "r"((int)row0), "r"(stage)
            : "memory");
}

// That lane: until all but `LEFT` of its copies have read their tiles; and until all have written.
template <int LEFT>
__device__ __forceinline__ void sent_read()
{
    if (elect_one()) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(LEFT) : "memory");
    __syncwarp();
}
__device__ __forceinline__ void sent_all()
{
    if (elect_one()) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// x += scale times the tile that is there.
template <int DT>
__device__ __forceinline__ void add_tile(uint32_t stage, int lane, float scale, float (&x)[32], const Matrix16& D, int64_t row0, int64_t col0)
{
    load_tile16(stage, lane, D, row0, col0);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t w[4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(tile16_at(stage, lane, i)) : "memory");
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float a, b;
            widen2<DT>(w[j], a, b);
            x[8 * i + 2 * j] += scale * a;
            x[8 * i + 2 * j + 1] += scale * b;
        }
    }
    __syncwarp();
}

// ------------------------------------------------------------------ a kernel of tiles
//
// One thread copies operand tiles into the ring, one issues the products, eight warps finish a tile while the next
// is multiplied: the frame of a persistent kernel whose tiles W describes:
//   range(worker, workers, i, end, step)    the tiles of a block or pair
//   Item item(int)                          where a tile is; Item::kb: its inner blocks, at least one
//   uint32_t bytes(Item)                    what a stage's copies bring, to both blocks of a pair
//   aside(lane)                             without a scout: what that warp does
//   kScout, bool begin(Item, Seen&)         true: a warp of its own finds the items and waits for what they wait for
//                                           (false: given up), ahead of the others, which take them from a queue
//   queue_ns()                              bound on their wait for an item there
//   load(Item, kb, a, b, bar, rank)         those copies
//   a_mn(Item, kb), b_mn(Item, kb), idesc(Item, kb)   how a stage's operands lie, and the product's descriptor
//   prepare(Item, quad, half, rank, lane, Ahead&)      what a tile's end may load before its products are done
//   finish(Item, Ahead&, acc, quad, half, stage, rank, lane)   TMEM lanes 32 quad on; alternate 32 columns a half
//   done(Item)                                         by each of those warps after it
//   gave_up()                                          by a thread whose wait ran out
// CG = 2: the two blocks of a cluster form one 256 x BN tile: each stages 128 rows of A and BN / 2 of B, the first
// one issues products that read both, and each keeps the accumulators of its own 128 rows.  CG = 1: 128 x BN.

// mbar_wait with the clock read rarely: reading it twice before the first try costs more than most waits here take.
__device__ __forceinline__ bool stage_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns = kGemmWaitNs)
{
    for (int i = 0; i < 8; ++i)
        if (mbar_try(bar, parity)) return true;
    return mbar_wait(bar, parity, limit_ns);
}

template <int CG, int BN>
struct Tiles {
    using S = GemmShape<CG, BN>;
    uint32_t base, epi0, full0, empty0, acc_full0, acc_empty0, queue_full0, queue_empty0, queue0, tmem, rank;
    int warp, lane;
    static constexpr int kQueue = 4, kItemBytes = 112;
    static constexpr int kScoutSmem = S::kSmem + kQueue * (kItemBytes + 16);     // with the queue

    template <bool SCOUT = false>
    __device__ __forceinline__ void open(unsigned char* smem_raw)
    {
        const uint32_t raw = (uint32_t)__cvta_generic_to_shared(smem_raw);
        base = (raw + 1023u) & ~1023u;
        epi0 = base + S::kStages * S::kStageBytes;
        full0 = epi0 + kEpiWarps * kEpiBytes;
        empty0 = full0 + 8 * S::kStages;
        acc_full0 = empty0 + 8 * S::kStages;
        acc_empty0 = acc_full0 + 16;
        const uint32_t tmem_slot = acc_empty0 + 16;
        queue0 = (full0 + 256 + 15) & ~15u;
        queue_full0 = queue0 + kQueue * kItemBytes;
        queue_empty0 = queue_full0 + 8 * kQueue;
        warp = threadIdx.x >> 5;
        lane = threadIdx.x & 31;
        rank = CG == 2 ? cluster_rank() : 0;
        if (warp == 0 && lane == 0) {
            for (int i = 0; i < S::kStages; ++i) {
                mbar_init(full0 + 8 * i, 1);
                mbar_init(empty0 + 8 * i, 1);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(acc_full0 + 8 * i, 1);
                mbar_init(acc_empty0 + 8 * i, kEpiWarps * CG);
            }
            if constexpr (SCOUT) {
                for (int i = 0; i < kQueue; ++i) {
                    mbar_init(queue_full0 + 8 * i, 1);
                    mbar_init(queue_empty0 + 8 * i, kEpiWarps + 1 + (rank == 0));
                }
            }
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
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
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tmem_slot));
    }

    // Item number `tile` of this block, to every lane that calls; one of them says that the warp has it.
    template <class W>
    __device__ __forceinline__ bool take(const W& work, int i, uint32_t tile, typename W::Item& I, bool whole_warp) const
    {
        if constexpr (W::kScout) {
            const uint32_t slot = tile % kQueue, at = queue0 + slot * kItemBytes;
            bool there = stage_wait(queue_full0 + 8 * slot, (tile / kQueue) & 1, work.queue_ns());
            // a warp has the item or gives up as one: the item may come as some lanes' waits run out, and the others
            // would wait for them below
            if (whole_warp) there = __all_sync(0xFFFFFFFFu, there);
            if (!there) return false;
            uint32_t w[kItemBytes / 4];
#pragma unroll
            for (int j = 0; j < kItemBytes / 16; ++j)
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[4 * j]), "=r"(w[4 * j + 1]), "=r"(w[4 * j + 2]), "=r"(w[4 * j + 3]) : "r"(at + 16 * j) : "memory");
            static_assert(sizeof(I) == kItemBytes, "an item's size");
            memcpy(&I, w, sizeof(I));
            if (whole_warp) __syncwarp();
            if (!whole_warp || lane == 0) mbar_arrive(queue_empty0 + 8 * slot);
        } else {
            I = work.item(i);
        }
        return true;
    }

    template <class W>
    __device__ __forceinline__ void run(const W& work, uint32_t* error)
    {
        int first, end, step;
        work.range((int)(blockIdx.x / CG), (int)(gridDim.x / CG), first, end, step);
        bool ok = true;
        if (warp == 0) {
            // ---- producer: one thread
            if (elect_one()) {
                uint32_t k = 0, tile = 0;
                for (int i = first; i < end && ok; i += step, ++tile) {
                    typename W::Item I;
                    ok = take(work, i, tile, I, false);
                    if (!ok) break;
                    const uint32_t bytes = work.bytes(I);
                    for (int kb = 0; kb < I.kb; ++kb, ++k) {
                        const uint32_t s = k % S::kStages, use = k / S::kStages;
                        if (use > 0 && !stage_wait(empty0 + 8 * s, (use - 1) & 1)) {
                            ok = false;
                            break;
                        }
                        const uint32_t a = base + s * S::kStageBytes;
                        uint32_t bar = full0 + 8 * s;
                        if (rank == 0) mbar_arrive_expect_tx(bar, bytes);
                        if constexpr (CG == 2) bar = leader_address(bar);
                        work.load(I, kb, a, a + S::kABytes, bar, (int)rank);
                    }
                }
            }
        } else if (warp == 1) {
            // ---- products: one thread of the leading block
            if (rank == 0 && elect_one()) {
                uint32_t k = 0, tile = 0;
                for (int i = first; i < end && ok; i += step, ++tile) {
                    typename W::Item I;
                    ok = take(work, i, tile, I, false);
                    if (!ok) break;
                    const uint32_t acc = tile & 1, use = tile >> 1;
                    if (use > 0 && !stage_wait(acc_empty0 + 8 * acc, (use - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    for (int kb = 0; kb < I.kb; ++kb, ++k) {
                        const uint32_t s = k % S::kStages;
                        if (!stage_wait(full0 + 8 * s, (k / S::kStages) & 1)) {
                            ok = false;
                            break;
                        }
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        const uint32_t a = base + s * S::kStageBytes;
                        const bool a_mn = work.a_mn(I, kb), b_mn = work.b_mn(I, kb);
                        const uint32_t idesc = work.idesc(I, kb);
                        // 16 inner elements: 32 bytes along K, two groups of eight K rows along MN
                        const uint64_t sa = a_mn ? 2048 >> 4 : 32 >> 4, sb = b_mn ? 2048 >> 4 : 32 >> 4;
                        const uint64_t da = smem_desc(a, a_mn), db = smem_desc(a + S::kABytes, b_mn);
#pragma unroll
                        for (int j = 0; j < kBK / 16; ++j)
                            mma_f16<CG>(tmem + acc * BN, da + sa * j, db + sb * j, idesc, kb > 0 || j > 0);
                        mma_commit<CG>(empty0 + 8 * s);
                    }
                    if (!ok) break;
                    mma_commit<CG>(acc_full0 + 8 * acc);
                }
            }
        } else if (warp == 3) {
            // ---- scout: one thread
            if constexpr (!W::kScout) {
                work.aside(lane);
            } else {
                if (lane == 0) {
                    typename W::Seen seen = {};
                    uint32_t tile = 0;
                    for (int i = first; i < end && ok; i += step, ++tile) {
                        const uint32_t slot = tile % kQueue, use = tile / kQueue, at = queue0 + slot * kItemBytes;
                        const typename W::Item I = work.item(i);
                        if (use > 0 && !stage_wait(queue_empty0 + 8 * slot, (use - 1) & 1)) {
                            ok = false;
                            break;
                        }
                        uint32_t w[kItemBytes / 4];
                        memcpy(w, &I, sizeof(I));
#pragma unroll
                        for (int j = 0; j < kItemBytes / 16; ++j)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + 16 * j), "r"(w[4 * j]), "r"(w[4 * j + 1]), "r"(w[4 * j + 2]), "r"(w[4 * j + 3]) : "memory");
                        ok = work.begin(I, seen);
                        if (!ok) break;
                        mbar_arrive(queue_full0 + 8 * slot);
                    }
                }
            }
        } else if (warp >= 4) {
            // ---- epilogue: warp w reads TMEM lanes 32 (w % 4) on; the two warps of a lane group take alternate
            // columns
            const int quad = warp & 3, half = (warp - 4) >> 2;
            const uint32_t stage = epi0 + (warp - 4) * kEpiBytes;
            const uint32_t acc_empty_leader = CG == 2 ? leader_address(acc_empty0) : acc_empty0;
            uint32_t tile = 0;
            for (int i = first; i < end && ok; i += step, ++tile) {
                const uint32_t acc = tile & 1, use = tile >> 1;
                typename W::Item I;
                ok = take(work, i, tile, I, true);
                if (!ok) break;
                typename W::Ahead ahead;
                work.prepare(I, quad, half, (int)rank, lane, ahead);
                ok = stage_wait(acc_full0 + 8 * acc, use & 1);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                work.finish(I, ahead, tmem + acc * BN + ((uint32_t)(quad * 32) << 16), quad, half, stage, (int)rank, lane);
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CG == 2) arrive_cluster(acc_empty_leader + 8 * acc);
                    else mbar_arrive(acc_empty0 + 8 * acc);
                }
                work.done(I);
            }
            sent_all();          // the block's memory outlives the copies from it
        }
        if (!ok) {
            // A wait ran out: say so, and give copies and products in flight time to end before the block's memory
            // is given back.
            atomicOr(error, 1u);
            work.gave_up();
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
};

// ------------------------------------------------------------------ aligned copies

// Rows copied to rows of `ld` elements that start on 16 bytes (src NULL: nothing to copy).
struct AlignJob {
    const uint16_t* src;
    uint16_t* dst;
    int64_t ld_src, ld, rows, cols;
};

// Block b of n, 256 threads: eight elements a thread at a time.
__device__ __forceinline__ void align_rows(const AlignJob& J, int b, int n)
{
    const int64_t per_row = (J.cols + 7) / 8, total = J.rows * per_row;
    for (int64_t i = (int64_t)b * 256 + threadIdx.y * blockDim.x + threadIdx.x; i < total; i += (int64_t)n * 256) {
        const int64_t row = i / per_row, col = (i - row * per_row) * 8;
        const uint16_t* p = J.src + row * J.ld_src + col;
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t lo = col + 2 * j < J.cols ? p[2 * j] : 0u, hi = col + 2 * j + 1 < J.cols ? p[2 * j + 1] : 0u;
            w[j] = lo | (hi << 16);
        }
        *reinterpret_cast<uint4*>(J.dst + row * J.ld + col) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// ------------------------------------------------------------------ few rows

__device__ __forceinline__ uint32_t word(const uint4& v, int j) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; }

// acc[m][c] += eight products of row m of x and row c of W, U times.  Loads first, none of them behind a
// branch.
template <int DT, int U, int ROWS, int C>
__device__ __forceinline__ void few_eights(const uint16_t* const (&x)[ROWS], const uint16_t* const (&w)[C], int64_t k, int64_t step, F2 (&acc)[ROWS][C])
{
    uint4 wv[U][C], xv[U][ROWS];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int c = 0; c < C; ++c) wv[u][c] = __ldcs(reinterpret_cast<const uint4*>(w[c] + k + u * step));
#pragma unroll
        for (int m = 0; m < ROWS; ++m) xv[u][m] = *reinterpret_cast<const uint4*>(x[m] + k + u * step);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            F2 f[C];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float a, b;
                widen2<DT>(word(wv[u][c], j), a, b);
                f[c] = pair(a, b);
            }
#pragma unroll
            for (int m = 0; m < ROWS; ++m) {
                float a, b;
                widen2<DT>(word(xv[u][m], j), a, b);
#pragma unroll
                for (int c = 0; c < C; ++c) acc[m][c] = fma(pair(a, b), f[c], acc[m][c]);
            }
        }
}

// ------------------------------------------------------------------ host

inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t up(int64_t a, int64_t b) { return div_up(a, b) * b; }

// A matrix as an operand: `rows` x `inner` (M or N by K) in 16 bits; mn: stored with its rows
// along memory (inner x rows in memory).
struct Operand {
    const void* p;
    int64_t rows, inner, ld;
    bool mn;
};

inline bool tma_ready(const void* p, int64_t ld) { return aligned(p, 16) && ld % 8 == 0; }

constexpr int kGb300Sms = 152;

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeFn encode_fn()
{
    static EncodeFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

inline zero_status_t encode_box(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int64_t ld, int dtype16, int box_rows, int box_cols,
                                const char* who)
{
    EncodeFn fn = encode_fn();
    if (!fn) return fail(ZERO_ECUDA, std::string(who) + ": the driver has no cuTensorMapEncodeTiled");
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    const cuuint32_t unit[2] = {1, 1};
    const CUresult r = fn(map, dtype16 == ZERO_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                          const_cast<void*>(p), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ZERO_OK : fail(ZERO_ECUDA, std::string(who) + ": a tensor map was refused (" + std::to_string((int)r) + ")");
}

inline zero_status_t encode(CUtensorMap* map, const Operand& o, int dtype16, int box_rows, const char* who)
{
    return encode_box(map, o.p, o.mn ? o.inner : o.rows, o.mn ? o.rows : o.inner, o.ld, dtype16, o.mn ? kBK : box_rows, 64, who);
}

inline int grid_of(int64_t items, int sms, int per_sm) { return (int)std::max<int64_t>(1, std::min<int64_t>(div_up(items, 256), (int64_t)sms * per_sm)); }

inline int vec_flag(const void* p, int64_t ld, int flag) { return p && aligned(p, 16) && ld % 8 == 0 ? flag : 0; }

}  // namespace
}  // namespace zero
