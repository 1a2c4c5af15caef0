// zero_muon.cu -- an optimizer whose update of a matrix is orthogonalised (zero_muon_*):
//   g = sum of the ranks' contributions / (N_d loss_scale);  m' = mu m + (1 - mu) g
//   u = mu m' + (1 - mu) g (nesterov), or m';  X = u / (||u||_F + eps)
//   X <- (a I + b G + c G^2) X, G = X X^T, `steps` times (a Newton-Schulz iteration for the polar factor; X^T X from
//   the right where X has more rows than columns)
//   p <- p - lr wd p;  p <- p - lr s X
//
// A pass over the contributions forms m' and the norms, one over the momentum the first X; then each iteration is three
// products on the tensor cores: G and the polynomial of it, of which only the upper triangle's tiles are multiplied and
// kept, and the polynomial times X.  Nothing is transposed in memory: a tensor map takes X, or a symmetric matrix's tile
// in place of the one across the diagonal, along its rows or along its columns.  Where every matrix is large, the first
// two iterations are one (launch_rest).  All products of all matrices are one cooperative launch: a matrix's next
// product begins when the one before it is complete, whatever the other matrices do, so that no round of tiles has to be
// full.  The last product's tiles go into the parameters and are never stored.
//
// Operands are fp16 whatever the gradients' type, times powers of two that keep them in its range (the iterates' are
// bounded: ||X||_2 <= 1 at first, and the coefficients give the rest).  Rounding to bf16's 8 bits costs 1 to 3 % of the
// result, as small singular values grow by a^steps (485) and what rounding adds to them grows with them; fp16's 11 bits
// 0.13 to 0.4 %, and with the first iterates as sums of two fp16 numbers (the products take the first; a X, which is
// nearly all of small singular values' growth, both) 0.1 to 0.3 % (2-norm, dense matrices with sides of 64 and more).  One
// direction over 1 % of noise, 512 x 512: 0.26 % instead of 2.7, for which the second number is there.  Few singular values
// have up to 1.1 % either way: 3 x 512, or 4 rows of 256 that are not zero.  tf32 has fp16's 11 bits at half its rate.
// Sums are fp32.
//
// Measured on one GB300: two layers of a 2048-wide GPT's matrices (101M elements) from 16 contributions 2,913 to 2,978
// us: the contributions 575 (7.0 TB/s), the first X 177 (6.8 TB/s), the products 1,900 as long as the clocks hold; a 4096 x 4096
// and an 11008 x 4096 matrix from 8 3,012 to 3,112; three layers 256 wide from four 131, 16 products of 5.6 us one after another.
// The products are bound by power: of the library's fp16 products of normal numbers (1,629 TFLOP/s sustained; 1,731 in
// bf16) they make 0.9, and the tensor cores are busy 81 % of the cycles.
#include <cmath>
#include <cstring>
#include <functional>
#include <initializer_list>
#include <memory>
#include <utility>
#include <vector>

#include "zero_mma.cuh"

namespace zero {
namespace {

// Set by a kernel whose bounded wait ran out (zero_operators_check reads and clears it).
__device__ uint32_t g_muon_error;

constexpr int kThreads = 256;
// Elements of a matrix that a block takes at a time, eight a thread.  Blocks take neighbouring ones in turn, so that
// what runs at one time reads a few MB of each contribution: with 32768 in a row the contributions' pages are too many
// (16 of 100M elements: 895 us; with 8192 816).
constexpr int kChunk = 8 * kThreads;
// Blocks an SM of the passes over the elements: as many as run at one time.  With six of the first pass, of which five
// run, 16 contributions of 50M elements took 360 us instead of 304 (6.6 TB/s).
constexpr int kReduceBlocks = 5, kStartBlocks = 6;
constexpr int kStateBlock = 256;          // each matrix's momentum starts on a multiple of it
constexpr int kRowElems = 16;             // rows of X and of the symmetric matrices are a multiple of it: 32 bytes
constexpr int kSquares = 4;               // symmetric matrices beside each X
constexpr int kMaxPhases = 32;            // products of a step, at most 25
constexpr int kTwice = 2;                 // iterations whose X is the sum of two fp16 numbers
constexpr int kPairSide = 128;            // smaller sides from which the first two iterations are one
constexpr float kLow = 2048.0f;           // the second of them is stored times this

struct MuonState {
    uint32_t flag;          // the open step's gradients are not finite
    uint32_t cur;           // the momentum's current half
    uint32_t last_skipped;
    uint32_t closed;        // blocks of the last pass that are done
    int64_t t, skipped, finished;
    uint32_t timeout;       // a wait of a step ran out since the last read, and its parameters may be partly moved
};
static_assert(sizeof(MuonState) <= 256, "MuonState fits its slot");

// A matrix's tensor maps.  Along K and along the rows of operands: X's two buffers, the symmetric matrices; to write
// tiles of 32 x 32: the same and X's low part.
enum { kMapX = 0, kMapXAcross = 2, kMapSquare = 4, kMapSquareAcross = 4 + kSquares, kMapOutX = 4 + 2 * kSquares,
       kMapOutLow = kMapOutX + 2, kMapOutSquare = kMapOutX + 3, kMaps = kMapOutSquare + kSquares };
static_assert(kMaps <= 32, "a bit a map");

struct alignas(128) MuonTensor {
    CUtensorMap map[kMaps];
    uint16_t *x[2], *low;        // rows x ldx
    uint16_t* square[kSquares];  // m x ldm
    float* p;                    // NULL: no parameters
    uint16_t *p16, *update;      // may be NULL
    int64_t at;                  // its first momentum
    float aspect, rms;           // factors of the update
    int32_t rows, cols, m, ldx, ldm;
    int32_t wide;                // rows <= cols: G = X X^T
    int32_t vec_g, vec_p;        // 16-byte accesses to the contributions; four elements at once of p, p16 and update
    int32_t chunks;              // of the first pass
    int32_t tiles[2];            // of a symmetric product, and of one with X
};

// A piece of a matrix's elements, or a tile of it (m << 16 | n).
struct Piece {
    int32_t tensor, at;
};

struct MuonParams {
    MuonTensor* tensors;
    const Piece* pieces;
    const void* const* grads;    // [tensor][n_d]
    float* momentum[2];
    MuonState* st;
    DevState* plan;              // a sharded step that this one is part of, or NULL
    double* slots;               // [piece of the first pass] sums of squares
    float* scale;                // [tensor] 1 / (norm + eps)
    uint32_t* tickets;           // [tensor]
    uint32_t* counters;          // [tensor][kMaxPhases]: warps that have stored their part of a product's tile
    int32_t n_counters;
    int32_t count, n_d, nesterov;
    float inv, mu, nu, sigma;    // nu = 1 - mu; sigma: X's factor in fp16
    double eps;
};

__device__ __forceinline__ float contribution_scale(const MuonParams& P)
{
    if (!P.plan) return P.inv;
    const volatile DevState* plan = P.plan;
    return __double2float_rn(__ddiv_rn(1.0, (double)P.n_d * plan->scale));
}

__device__ __forceinline__ float ahead(float m0, float m1, const MuonParams& P)
{
    // mu m' + (1 - mu) g, (1 - mu) g = m' - mu m
    return P.nesterov ? fmaf(P.mu, m1, fmaf(-P.mu, m0, m1)) : m1;
}

// ------------------------------------------------------------------ the contributions into the momentum

// Eight elements from e on (n of them there): the sum of the contributions.
template <int DT>
__device__ __forceinline__ void sum_contributions(const void* const* grads, int n_d, int64_t e, int n, bool vec, float (&g)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = 0.0f;
    auto add8 = [&](const uint4& w) {
        float x[8];
        widen2<DT>(w.x, x[0], x[1]);
        widen2<DT>(w.y, x[2], x[3]);
        widen2<DT>(w.z, x[4], x[5]);
        widen2<DT>(w.w, x[6], x[7]);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] += x[j];
    };
    int r = 0;
    if (vec && n == 8) {
        for (; r + 8 <= n_d; r += 8) {
            uint4 w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(grads[r + i]) + e));
#pragma unroll
            for (int i = 0; i < 8; ++i) add8(w[i]);
        }
        if (r + 4 <= n_d) {
            uint4 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(grads[r + i]) + e));
#pragma unroll
            for (int i = 0; i < 4; ++i) add8(w[i]);
            r += 4;
        }
        for (; r < n_d; ++r) add8(__ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(grads[r]) + e)));
    } else {
        for (; r < n_d; ++r) {
            const uint16_t* p = static_cast<const uint16_t*>(grads[r]) + e;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) g[j] += widen1<DT>(p[j]);
        }
    }
}

// A block's sum of squares of a matrix goes to the slot of its first piece of it; the last of the blocks that have any
// sums them, in order.
template <int DT>
__global__ void __launch_bounds__(kThreads, kReduceBlocks) muon_reduce_kernel(const __grid_constant__ MuonParams P)
{
    after_earlier_work();
    __shared__ double warp_sum[kThreads / 32];
    __shared__ const void* grads[ZERO_MAX_RANKS];
    __shared__ bool last;
    const uint32_t cur = *(const volatile uint32_t*)&P.st->cur;
    const float *from = P.momentum[cur & 1];
    float* to = P.momentum[(cur & 1) ^ 1];
    const float inv = contribution_scale(P);
    int i = blockIdx.x;
    Piece next = P.pieces[min(i, P.count - 1)];
    while (i < P.count) {
        // every piece of this block of one matrix
        const int tensor = next.tensor, first = i;
        const MuonTensor& T = P.tensors[tensor];
        const int64_t elems = (int64_t)T.rows * T.cols, at = T.at;
        const int chunks = T.chunks, head = i - next.at;
        const bool vec = T.vec_g;
        __syncthreads();
        for (int r = threadIdx.x; r < P.n_d; r += kThreads) grads[r] = P.grads[(int64_t)tensor * P.n_d + r];
        __syncthreads();
        float sum = 0.0f;
        while (i < P.count && next.tensor == tensor) {
            const int64_t e = (int64_t)next.at * kChunk + threadIdx.x * 8;
            const int n = (int)max((int64_t)0, min((int64_t)8, elems - e));
            i += gridDim.x;
            next = P.pieces[min(i, P.count - 1)];
            if (n <= 0) continue;
            // the momentum's rows of eight are whole: it is padded
            const float4* q = reinterpret_cast<const float4*>(from + at + e);
            const float4 a = __ldcs(q), b = __ldcs(q + 1);
            float g[8];
            sum_contributions<DT>(grads, P.n_d, e, n, vec, g);
            const float m0[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            float m1[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                m1[j] = j < n ? fmaf(P.mu, m0[j], P.nu * (g[j] * inv)) : 0.0f;
                const float u = j < n ? ahead(m0[j], m1[j], P) : 0.0f;
                sum = fmaf(u, u, sum);
            }
            float4* o = reinterpret_cast<float4*>(to + at + e);
            __stcs(o, make_float4(m1[0], m1[1], m1[2], m1[3]));
            __stcs(o + 1, make_float4(m1[4], m1[5], m1[6], m1[7]));
        }
        const int sharers = min(chunks, (int)gridDim.x);
        const double s = block_sum_fixed<kThreads>((double)sum, warp_sum);
        if (threadIdx.x == 0) {
            P.slots[first] = s;
            __threadfence();
            last = atomicAdd(&P.tickets[tensor], 1u) == (uint32_t)sharers - 1;
        }
        __syncthreads();
        if (!last) continue;
        __threadfence();
        const volatile double* slots = P.slots + head;
        double x = 0.0;
        for (int k = threadIdx.x; k < sharers; k += kThreads) x += slots[k];
        const double norm2 = block_sum_fixed<kThreads>(x, warp_sum);
        if (threadIdx.x == 0) {
            P.tickets[tensor] = 0;
            P.scale[tensor] = (float)(1.0 / (sqrt(norm2) + P.eps));
            if (!isfinite(norm2)) atomicOr(P.plan ? &P.plan->flag : &P.st->flag, 1u);
        }
    }
}

// ------------------------------------------------------------------ the first X

__device__ __forceinline__ void load_floats(const float* p, float (&x)[8])
{
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

__device__ __forceinline__ void two_halves(const float (&x)[8], uint32_t (&hi)[4], uint32_t (&low)[4])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float a, b;
        hi[j] = narrow2<ZERO_FP16>(x[2 * j], x[2 * j + 1]);
        widen2<ZERO_FP16>(hi[j], a, b);
        low[j] = narrow2<ZERO_FP16>((x[2 * j] - a) * kLow, (x[2 * j + 1] - b) * kLow);
    }
}

// This thread's eight columns in piece `at` of a matrix, cut as X is laid out: where they are in the matrix and in X,
// and how many are there (0: none of it).
struct Eight {
    int64_t e, x;
    int n;
};

__device__ __forceinline__ Eight eight_at(const MuonTensor& T, int at)
{
    const int64_t groups = T.ldx / 8, i = (int64_t)at * kThreads + threadIdx.x;
    Eight E{i * 8, i * 8, 8};
    if (i >= T.rows * groups) {
        E.n = 0;
    } else if (T.cols != T.ldx) {
        const int64_t row = i / groups, col = (i - row * groups) * 8;
        E.e = row * T.cols + col;
        E.n = (int)max((int64_t)0, min((int64_t)8, T.cols - col));
    }
    return E;
}

__global__ void __launch_bounds__(kThreads, kStartBlocks) muon_start_kernel(const __grid_constant__ MuonParams P)
{
    after_earlier_work();
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < P.n_counters; i += gridDim.x * kThreads) P.counters[i] = 0;
    const uint32_t cur = *(const volatile uint32_t*)&P.st->cur;
    Piece next = P.pieces[min((int)blockIdx.x, P.count - 1)];
    for (int i = blockIdx.x; i < P.count; i += gridDim.x) {
        const Piece piece = next;
        next = P.pieces[min(i + (int)gridDim.x, P.count - 1)];
        const MuonTensor& T = P.tensors[piece.tensor];
        const Eight E = eight_at(T, piece.at);
        if (E.n == 0) continue;
        const bool vec = T.cols % 8 == 0;
        const float scale = P.scale[piece.tensor];
        const float *old = P.momentum[cur & 1] + T.at + E.e, *now = P.momentum[(cur & 1) ^ 1] + T.at + E.e;
        float m0[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f}, m1[8], x[8];
        if (vec) {
            load_floats(now, m1);
            if (P.nesterov) load_floats(old, m0);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                m1[j] = j < E.n ? now[j] : 0.0f;
                m0[j] = j < E.n && P.nesterov ? old[j] : 0.0f;
            }
        }
        uint32_t hi[4], low[4];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = (ahead(m0[j], m1[j], P) * scale) * P.sigma;
        two_halves(x, hi, low);
        *reinterpret_cast<uint4*>(T.x[0] + E.x) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(T.low + E.x) = make_uint4(low[0], low[1], low[2], low[3]);
    }
}

// ------------------------------------------------------------------ the parameters

// Is the step left out?  A wait that runs out says so to it too (gave_up), and to the steps that follow until it is read.
__device__ __forceinline__ bool left_out(const MuonState* st, const DevState* plan)
{
    if (!plan) {
        const volatile MuonState* s = st;
        return (s->flag | s->timeout) != 0;
    }
    const volatile DevState* p = plan;
    return (p->flag | p->error) != 0;
}

// By the last block, when every block has read the flag.
__device__ __forceinline__ void close_step(MuonState* state, bool skip)
{
    volatile MuonState* st = state;
    st->closed = 0;
    st->flag = 0;
    st->finished = st->finished + 1;
    st->last_skipped = skip ? 1u : 0u;
    if (skip) {
        st->skipped = st->skipped + 1;
    } else {
        st->t = st->t + 1;
        st->cur = (st->cur & 1) ^ 1;
    }
}

// A step without elements.
__global__ void __launch_bounds__(32) muon_close_kernel(MuonState* st, DevState* plan)
{
    after_earlier_work();
    if (threadIdx.x == 0) close_step(st, left_out(st, plan));
}

__device__ __forceinline__ uint16_t narrow_to(float x, bool bf) { return bf ? narrow1<ZERO_BF16>(x) : narrow1<ZERO_FP16>(x); }
__device__ __forceinline__ uint2 narrow_to(const float4& x, bool bf)
{
    return bf ? make_uint2(narrow2<ZERO_BF16>(x.x, x.y), narrow2<ZERO_BF16>(x.z, x.w)) : make_uint2(narrow2<ZERO_FP16>(x.x, x.y), narrow2<ZERO_FP16>(x.z, x.w));
}

// p - decay p - step x
__device__ __forceinline__ float moved(float p, float x, float step, float decay) { return fmaf(-step, x, fmaf(-decay, p, p)); }

// ------------------------------------------------------------------ the products

// Rows of a box of an operand taken along K.
constexpr int box_rows(int bn) { return bn == 64 ? 64 : 128; }

// X X^T (or X^T X); a product of two symmetric matrices that commute, so that it is one too; one times X.
enum { kGram = 0, kSquare = 1, kNext = 2 };

// One product of every matrix: out = scale acc + lin[0] add0 + lin[1] add1 + diag I.  Symmetric matrices by their
// slots; kNext's addends are X and its low part.
struct Op {
    int32_t kind, src;           // src: X's buffer that is read
    int32_t left, right, out;    // operands and result; kNext: left is the polynomial
    int32_t adds, add[2];
    int32_t keep_low;            // kNext: the successor's low part is wanted
    int32_t final;               // kNext: the result is the update, for the parameters
    float scale, lin[2], diag;
};

struct ProductParams {
    const MuonTensor* tensors;
    const Piece* tiles;          // each worker's, in the order of the products: tensor | product << 16
    const int32_t* bounds;       // [worker][kMaxPhases]: where its tiles of each product begin
    uint32_t* counters;
    MuonState* st;
    DevState* plan;              // a sharded step that this one is part of, or NULL
    int32_t how, bf;             // ZERO_MUON_SCALE_*; the 16-bit type is bf16
    float lr, decay;             // lr weight_decay
    uint64_t wait_ns;            // bound on a wait for the product before
    int32_t first, last;         // products that are made
    Op ops[kMaxPhases];          // ops[i - first] is product i
};

__device__ __forceinline__ uint32_t load_relaxed(const uint32_t* p)
{
    uint32_t v;
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

template <int CG, int BN>
struct MuonWork {
    const ProductParams& P;
    struct alignas(16) Item {
        const uint32_t* before;  // the matrix's counter of the product before, or NULL
        uint32_t* counter;       // and of this one
        const CUtensorMap* maps; // the matrix's
        const uint16_t* add[2];
        int32_t ld, rows, cols;  // of the result and the addends
        int32_t m, n, kb, kind, tensor;
        uint32_t want;           // of `before`
        float scale, lin[2], diag;
        int8_t adds, keep_low, final;
        int8_t a, b, out;        // maps: operands along K, or along their own rows where `along` says so; the result
        int8_t along;            // 1: a is, 2: b is
        int8_t square;           // 1: a, 2: b is symmetric: tiles below the diagonal are taken from above it
        int32_t reserved[2];
    };
    static constexpr bool kScout = true;

    __device__ __forceinline__ void range(int worker, int, int& i, int& end, int& step) const
    {
        i = P.bounds[worker * kMaxPhases + P.first];
        end = P.bounds[worker * kMaxPhases + P.last];
        step = 1;
    }

    __device__ __forceinline__ Item item(int i) const
    {
        const Piece t = P.tiles[i];
        const int tensor = t.tensor & 0xFFFF, phase = (t.tensor >> 16) - P.first;
        const MuonTensor& T = P.tensors[tensor];
        Item I;
        const Op& O = P.ops[phase];
        I.scale = O.scale;
        I.lin[0] = O.lin[0];
        I.lin[1] = O.lin[1];
        I.diag = O.diag;
        I.adds = (int8_t)O.adds;
        I.keep_low = (int8_t)O.keep_low;
        I.final = (int8_t)O.final;
        I.maps = T.map;
        I.tensor = tensor;
        I.m = t.at >> 16;
        I.n = t.at & 0xFFFF;
        I.kind = O.kind;
        I.counter = P.counters + tensor * kMaxPhases + phase;
        I.before = phase > 0 ? I.counter - 1 : nullptr;
        I.want = 0;
        if (phase > 0) I.want = (uint32_t)T.tiles[P.ops[phase - 1].kind == kNext] * (kEpiWarps * CG);
        const bool wide = T.wide;
        int inner = T.m;
        if (I.kind == kNext) {
            I.out = kMapOutX + (O.src ^ 1);
            I.add[0] = T.x[O.src];
            I.add[1] = T.low;
            I.ld = I.cols = T.ldx;
            I.rows = T.rows;
        } else {
            I.out = kMapOutSquare + O.out;
            I.add[0] = T.square[O.add[0]];
            I.add[1] = T.square[O.add[1]];
            I.ld = I.cols = T.ldm;
            I.rows = T.m;
        }
        if (I.kind == kGram) {
            I.a = I.b = (wide ? kMapX : kMapXAcross) + O.src;
            I.along = wide ? 0 : 3;
            I.square = 0;
            inner = wide ? T.cols : T.rows;
        } else if (I.kind == kSquare) {
            I.a = kMapSquare + O.left;
            I.b = kMapSquare + O.right;
            I.along = 0;
            I.square = 3;
        } else {
            I.a = wide ? kMapSquare + O.left : kMapX + O.src;
            I.b = wide ? kMapXAcross + O.src : kMapSquare + O.left;
            I.along = wide ? 2 : 0;
            I.square = wide ? 1 : 2;
        }
        I.kb = (inner + kBK - 1) / kBK;
        return I;
    }

    // Until every part of the product before is stored: a bounded wait.  A fence follows it.
    __device__ __forceinline__ bool wait_before(const Item& I) const
    {
        if (!I.before || load_relaxed(I.before) >= I.want) return true;
        const uint64_t t0 = global_ns();
        for (uint32_t i = 0; i < kWaitIterCap; ++i) {
            if (load_relaxed(I.before) >= I.want) return true;
            if (i % 16 == 15 && global_ns() - t0 > P.wait_ns) break;
        }
        return false;
    }

    // The tensor maps that a tile's copies take, written by the host into memory that may have held others.
    __device__ __forceinline__ static void see(const CUtensorMap* map)
    {
        asm volatile("fence.proxy.tensormap::generic.acquire.sys [%0], 128;" ::"l"(map) : "memory");
    }
    // What a block has waited for last, and the tensor maps that it has seen (a bit each, of the first matrices).
    struct Seen {
        static constexpr int kMatrices = 64;
        const uint32_t* before;
        uint32_t maps[kMatrices];
    };
    __device__ __forceinline__ bool begin(const Item& I, Seen& S) const
    {
        uint32_t use = 1u << I.a | 1u << I.b | 1u << I.out;
        if (I.square & 1) use |= 1u << (I.a + kSquares);
        if (I.square & 2) use |= 1u << (I.b + kSquares);
        if (I.keep_low) use |= 1u << kMapOutLow;
        if (I.tensor < Seen::kMatrices) {
            const uint32_t old = S.maps[I.tensor];
            S.maps[I.tensor] = old | use;
            use &= ~old;
        }
        for (; use; use &= use - 1) see(I.maps + (__ffs(use) - 1));
        if (I.before != S.before) {
            if (!wait_before(I)) return false;
            // with the writers' releases: what their copies wrote is read here, by loads and by copies
            asm volatile("fence.acq_rel.gpu;\n\tfence.proxy.async;" ::: "memory");
            S.before = I.before;
        }
        return true;
    }
    // One lane has sent the warp's tiles: once they are written, and so visible to it, its one release of them all.
    __device__ __forceinline__ void done(const Item& I) const
    {
        sent_all();
        if (elect_one()) asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(I.counter) : "memory");
    }

    // The scout's wait and what may keep it from the next.
    __device__ __forceinline__ uint64_t queue_ns() const { return P.wait_ns + kGemmWaitNs; }

    // Before this block counts itself as done (muon_product_kernel), so that what closes the step sees it.
    __device__ __forceinline__ void gave_up() const
    {
        atomicOr(&P.st->timeout, 1u);
        if (P.plan) atomicOr(&P.plan->error, 8u);
        __threadfence();
    }

    // Is an inner block below the diagonal block (kBM * CG wide) of a symmetric operand's rows from `row` on?
    __device__ __forceinline__ static bool below(int row, int kb) { return kb / (kBM * CG / kBK) < row / (kBM * CG); }

    __device__ __forceinline__ uint32_t bytes(const Item&) const { return CG * (kBM + BN / CG) * (kBK * 2); }
    __device__ __forceinline__ bool a_mn(const Item& I, int kb) const { return (I.along & 1) || ((I.square & 1) && below(I.m * (kBM * CG), kb)); }
    __device__ __forceinline__ bool b_mn(const Item& I, int kb) const { return (I.along & 2) || ((I.square & 2) && below(I.n * BN, kb)); }
    __device__ __forceinline__ uint32_t idesc(const Item& I, int kb) const
    {
        return (1u << 4) | ((a_mn(I, kb) ? 1u : 0u) << 15) | ((b_mn(I, kb) ? 1u : 0u) << 16) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)((kBM * CG) >> 4) << 24);
    }

    // ROWS rows of an operand: along K in boxes of kBox rows, along its own rows in boxes of 64
    static constexpr int kBox = box_rows(BN);
    template <int ROWS>
    __device__ __forceinline__ static void bring(const CUtensorMap* map, bool mn, uint32_t at, int row, int k, uint32_t bar)
    {
        if (mn) {
#pragma unroll
            for (int i = 0; i < ROWS / 64; ++i) tma_load_2d<CG>(at + i * (kBK * 128), map, row + 64 * i, k, bar);
        } else {
#pragma unroll
            for (int i = 0; i < ROWS / kBox; ++i) tma_load_2d<CG>(at + i * (kBox * kBK * 2), map, k, row + kBox * i, bar);
        }
    }

    __device__ __forceinline__ void load(const Item& I, int kb, uint32_t a, uint32_t b, uint32_t bar, int rank) const
    {
        const bool a_mn_ = a_mn(I, kb), b_mn_ = b_mn(I, kb);
        const int map_a = I.a + ((I.square & 1) && a_mn_ ? kSquares : 0), map_b = I.b + ((I.square & 2) && b_mn_ ? kSquares : 0);
        bring<kBM>(I.maps + map_a, a_mn_, a, (I.m * CG + rank) * kBM, kb * kBK, bar);
        bring<BN / CG>(I.maps + map_b, b_mn_, b, I.n * BN + rank * (BN / CG), kb * kBK, bar);
    }

    // ---- a tile's end.  The addends of a 32 x 32 part are loaded while the one before it is finished, the first
    // ones' while the products run: their latency, a microsecond, is otherwise most of a part's time.
    struct Ahead {
        uint4 v[2][4];
    };
    // Row `lane` of a 32 x 32 part: two loads of 32 bytes, as rows are of a multiple of 16 columns and start on 32 bytes.
    // A load touches 32 rows, but what it brings needs no turning through shared memory, which the products read all
    // the time (three layers 256 wide 147 -> 139 us).  From L2: other blocks write these buffers while this kernel runs.
    __device__ __forceinline__ static void fetch(uint4 (&v)[4], const uint16_t* p, const Item& L, int64_t row, int64_t col0)
    {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[2 * i] = v[2 * i + 1] = make_uint4(0u, 0u, 0u, 0u);
            if (row < L.rows && col0 + 16 * i < L.ld)
                asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                             : "=r"(v[2 * i].x), "=r"(v[2 * i].y), "=r"(v[2 * i].z), "=r"(v[2 * i].w), "=r"(v[2 * i + 1].x), "=r"(v[2 * i + 1].y),
                               "=r"(v[2 * i + 1].z), "=r"(v[2 * i + 1].w)
                             : "l"(p + row * L.ld + col0 + 16 * i)
                             : "memory");
        }
    }
    __device__ __forceinline__ static void add_row(const uint4 (&v)[4], float lin, float (&x)[32])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float a, b;
                widen2<ZERO_FP16>(word(v[i], j), a, b);
                x[8 * i + 2 * j] = fmaf(lin, a, x[8 * i + 2 * j]);
                x[8 * i + 2 * j + 1] = fmaf(lin, b, x[8 * i + 2 * j + 1]);
            }
    }

    __device__ __forceinline__ void fetch_adds(const Item& I, Ahead& A, int64_t row0, int c, int lane) const
    {
        const int adds = I.adds;
        if (adds > 0) fetch(A.v[0], I.add[0], I, row0 + lane, (int64_t)I.n * BN + c);
        if (adds > 1) fetch(A.v[1], I.add[1], I, row0 + lane, (int64_t)I.n * BN + c);
    }

    // The last product's end: x goes into the parameters, in fp32 through shared memory, so that a warp reads and writes
    // neighbours; the parameters of the next part are loaded as this one's are stored.
    struct Target {
        float* p;
        uint16_t *p16, *update;
        int32_t rows, cols;
        bool vec;
        float step;
    };
    __device__ __forceinline__ Target target(const Item& I) const
    {
        const MuonTensor& T = P.tensors[I.tensor];
        const float s = P.how == ZERO_MUON_SCALE_RMS ? T.rms : P.how == ZERO_MUON_SCALE_ASPECT ? T.aspect : 1.0f;
        return Target{T.p, T.p16, T.update, T.rows, T.cols, T.vec_p != 0, P.lr * s};
    }
    // Four parameters: row i * 4 + lane / 8 of the part, columns 4 (lane % 8) on.
    __device__ __forceinline__ static uint4 parameters(const Target& G, int64_t row0, int64_t col0, int i, int lane)
    {
        const int64_t row = row0 + i * 4 + (lane >> 3), col = col0 + (lane & 7) * 4;
        if (!G.p || row >= G.rows || col >= G.cols) return make_uint4(0u, 0u, 0u, 0u);
        return __ldcs(reinterpret_cast<const uint4*>(G.p + row * G.cols + col));
    }
    __device__ __forceinline__ static uint32_t turned_at(uint32_t stage, int row, int piece) { return stage + row * 128 + ((piece ^ (row & 7)) << 4); }

    __device__ __forceinline__ void apply(const Target& G, Ahead& A, bool more, int64_t row0, int64_t col0, int lane, uint32_t stage, const float (&x)[32]) const
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(turned_at(stage, lane, i)), "f"(x[4 * i]), "f"(x[4 * i + 1]), "f"(x[4 * i + 2]), "f"(x[4 * i + 3]) : "memory");
        __syncwarp();
        if (G.vec) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint4& w = A.v[i >> 2][i & 3];
                const int r = i * 4 + (lane >> 3);
                const int64_t row = row0 + r, col = col0 + (lane & 7) * 4;
                float4 z, p = make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
                asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(z.x), "=f"(z.y), "=f"(z.z), "=f"(z.w) : "r"(turned_at(stage, r, lane & 7)) : "memory");
                if (more) w = parameters(G, row0, col0 + 2 * kEpiCols, i, lane);
                if (row >= G.rows || col >= G.cols) continue;
                const int64_t e = row * G.cols + col;
                if (G.update) __stcs(reinterpret_cast<uint2*>(G.update + e), narrow_to(z, P.bf));
                if (!G.p) continue;
                p = make_float4(moved(p.x, z.x, G.step, P.decay), moved(p.y, z.y, G.step, P.decay), moved(p.z, z.z, G.step, P.decay), moved(p.w, z.w, G.step, P.decay));
                __stcs(reinterpret_cast<float4*>(G.p + e), p);
                if (G.p16) __stcs(reinterpret_cast<uint2*>(G.p16 + e), narrow_to(p, P.bf));
            }
        } else if (col0 + lane < G.cols) {
            // a column a lane; eight rows loaded before any is stored
            const int rows = (int)min((int64_t)32, G.rows - row0);
            for (int r0 = 0; r0 < rows; r0 += 8) {
                float p[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) p[j] = G.p && r0 + j < rows ? G.p[(row0 + r0 + j) * G.cols + col0 + lane] : 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (r0 + j >= rows) break;
                    const int64_t e = (row0 + r0 + j) * G.cols + col0 + lane;
                    float z;
                    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(z) : "r"(turned_at(stage, r0 + j, lane >> 2) + (lane & 3) * 4) : "memory");
                    if (G.update) G.update[e] = narrow_to(z, P.bf);
                    if (!G.p) continue;
                    const float q = moved(p[j], z, G.step, P.decay);
                    G.p[e] = q;
                    if (G.p16) G.p16[e] = narrow_to(q, P.bf);
                }
            }
        }
        __syncwarp();
    }

    __device__ __forceinline__ void finish_final(const Item& I, Ahead& A, uint32_t acc, int quad, int half, uint32_t stage, int rank, int lane) const
    {
        if (left_out(P.st, P.plan)) return;
        const Target G = target(I);
        const int64_t row0 = ((int64_t)I.m * CG + rank) * kBM + quad * 32;
        for (int c = half * kEpiCols; c < BN; c += 2 * kEpiCols) {
            const int64_t col0 = (int64_t)I.n * BN + c;
            if (col0 >= I.cols || row0 >= I.rows) break;
            float x[32];
            tmem_load32(acc + c, x);
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] *= I.scale;
            if (I.adds > 0) {
                // one or two steps in all: the addends and the parameters are loaded here
                fetch_adds(I, A, row0, c, lane);
                add_row(A.v[0], I.lin[0], x);
                if (I.adds > 1) add_row(A.v[1], I.lin[1], x);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (G.vec) A.v[i >> 2][i & 3] = parameters(G, row0, col0, i, lane);
            }
            apply(G, A, I.adds == 0 && c + 2 * kEpiCols < BN, row0, col0, lane, stage, x);
        }
    }

    __device__ __forceinline__ void prepare(const Item& I, int quad, int half, int rank, int lane, Ahead& A) const
    {
        if (I.final) {
            if (I.adds > 0) return;
            const Target G = target(I);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (G.vec) A.v[i >> 2][i & 3] = parameters(G, ((int64_t)I.m * CG + rank) * kBM + quad * 32, (int64_t)I.n * BN + half * kEpiCols, i, lane);
            return;
        }
        fetch_adds(I, A, ((int64_t)I.m * CG + rank) * kBM + quad * 32, half * kEpiCols, lane);
    }

    __device__ __forceinline__ void finish(const Item& I, Ahead& A, uint32_t acc, int quad, int half, uint32_t stage, int rank, int lane) const
    {
        if (I.final) {
            finish_final(I, A, acc, quad, half, stage, rank, lane);
            return;
        }
        const int64_t row0 = ((int64_t)I.m * CG + rank) * kBM + quad * 32;
        uint32_t turn = 0;
        for (int c = half * kEpiCols; c < BN; c += 2 * kEpiCols, turn ^= kTile16Bytes) {
            const int64_t col0 = (int64_t)I.n * BN + c;
            if (col0 >= I.cols || row0 >= I.rows) break;
            float x[32];
            tmem_load32(acc + c, x);
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] *= I.scale;
            if (I.adds > 0) add_row(A.v[0], I.lin[0], x);
            if (I.adds > 1) add_row(A.v[1], I.lin[1], x);
            if (c + 2 * kEpiCols < BN) fetch_adds(I, A, row0, c + 2 * kEpiCols, lane);
            // the warp's two tiles in turn, unless the low part needs one
            const uint32_t at = I.keep_low ? stage : stage + turn;
            if (I.keep_low) sent_read<0>();
            else sent_read<1>();
            if (I.kind != kNext && row0 == col0) {
#pragma unroll
                for (int j = 0; j < 32; ++j) x[j] += j == lane ? I.diag : 0.0f;
            }
            write_tile16<ZERO_FP16>(at, lane, x);
            send_tile16(at, I.maps + I.out, row0, col0);
            if (I.keep_low) {
#pragma unroll
                for (int j = 0; j < 32; ++j) x[j] = (x[j] - widen1<ZERO_FP16>(narrow1<ZERO_FP16>(x[j]))) * kLow;
                write_tile16<ZERO_FP16>(stage + kTile16Bytes, lane, x);
                send_tile16(stage + kTile16Bytes, I.maps + kMapOutLow, row0, col0);
            }
        }
    }
};

// Blocks wait for one another: a cooperative launch.
template <int CG, int BN>
__global__ void __cluster_dims__(CG, 1, 1) __launch_bounds__(kGemmThreads, 1) muon_product_kernel(const __grid_constant__ ProductParams P)
{
    extern __shared__ unsigned char smem_raw[];
    Tiles<CG, BN> T;
    T.template open<true>(smem_raw);
    after_earlier_work();
    T.run(MuonWork<CG, BN>{P}, &g_muon_error);
    if (threadIdx.x == 0 && atomicAdd(&P.st->closed, 1u) == gridDim.x - 1) {
        __threadfence();
        close_step(P.st, left_out(P.st, P.plan));
    }
}

}  // namespace

cudaError_t take_muon_error(uint32_t* word, void* stream) { return take_error_word(g_muon_error, word, static_cast<cudaStream_t>(stream)); }

}  // namespace zero

struct zero_muon {
    int n_d = 0, dtype16 = 0;
    std::vector<int64_t> rows, cols;
    int64_t elems = 0, state_elems = 0;
    int cg = 1, bn = 128;        // tiles of 128 x 64 or 128 x 128 on a block, or of 256 x 256 on a pair
    bool pair = false;
    std::vector<zero::Piece> chunks, groups, tiles;   // tiles: each worker's, in the order of the products
    std::vector<int32_t> bounds;
    int workers = 0;             // that the tiles are dealt to where every SM can be had
    int running = 0;             // the bound ones: as many as are resident at one time, or as the option says
    int64_t most_sms = 0;        // ZERO_MUON_OPT_SMS
    // the workspace's pieces
    int64_t at_tensors = 0, at_grads = 0, at_chunks = 0, at_groups = 0, at_tiles = 0, at_bounds = 0, at_counters = 0, at_slots = 0, at_scale = 0, at_tickets = 0,
            at_data = 0, bytes = 0;
    // bound buffers (caller-owned)
    bool bound = false;
    int device = -1;
    float* momentum[2] = {nullptr, nullptr};
    void* workspace = nullptr;
    // the sharded step (zero_plan::step_no) that zero_muon_check, zero_muon_step_with joined last
    int64_t checked_in = 0, stepped_in = 0;
    double checked_mu = 0.0;
    int64_t checked_flags = 0;
    int64_t wait_ns = (int64_t)zero::kGemmWaitNs;    // ZERO_MUON_OPT_WAIT_LIMIT_NS
};

namespace zero {
namespace {

// The symmetric matrices of an iteration, and where each is kept: G and the polynomial; for two iterations at once R1 =
// b G + c G^2, W = R1 G, the second's G and R, and Q = (a I + R1)(a' I + R2) - a a' I.
enum Role { kG, kPoly, kR1, kW, kG2, kR2, kQ, kRoles };
constexpr int kSlot[kRoles] = {0, 1, 1, 2, 3, 0, 2};

// What X and the symmetric matrices are multiplied by in fp16: powers of two that leave room below 65504.
struct Range {
    double sigma = 1.0, factor[kRoles];
    double of(Role r) const { return factor[r]; }
};

double power_below(double limit) { return std::exp2(std::floor(std::log2(limit))); }

// The largest of |f| on [0, hi], f(g) = k0 + k1 g + k2 g^2: at an end or where the slope is 0.
double largest(double k0, double k1, double k2, double hi)
{
    auto f = [&](double g) { return std::fabs(k0 + g * (k1 + g * k2)); };
    double m = std::max(f(0.0), f(hi));
    const double g = k2 != 0.0 ? -k1 / (2.0 * k2) : -1.0;
    return g > 0.0 && g < hi ? std::max(m, f(g)) : m;
}

// The largest of |a s + b s^3 + c s^5| on [0, hi].
double largest_step(const double* k, double hi)
{
    auto f = [&](double s) { return std::fabs(s * (k[0] + s * s * (k[1] + s * s * k[2]))); };
    double m = f(hi);
    // a + 3 b g + 5 c g^2 = 0, g = s^2
    const double root = 9.0 * k[1] * k[1] - 20.0 * k[0] * k[2];
    double g[2] = {-1.0, -1.0};
    if (k[2] == 0.0) {
        if (k[1] != 0.0) g[0] = -k[0] / (3.0 * k[1]);
    } else if (root >= 0.0) {
        g[0] = (-3.0 * k[1] - std::sqrt(root)) / (10.0 * k[2]);
        g[1] = (-3.0 * k[1] + std::sqrt(root)) / (10.0 * k[2]);
    }
    for (const double x : g)
        if (x > 0.0 && x < hi * hi) m = std::max(m, f(std::sqrt(x)));
    return m;
}

// Bounds of the singular values of all of them from the coefficients, with slack for rounding.  False: they grow too
// far.
bool find_range(const zero_muon_hyper_t& hyper, bool pair, Range* r)
{
    double hi = 1.0, x = 1.0, most[kRoles];
    for (double& m : most) m = 1e-6;
    auto see = [&](Role role, double v) { most[role] = std::max(most[role], std::fabs(v)); };
    for (int k = 0; k < hyper.steps; ++k) {
        const double* c = hyper.coefficients[k];
        see(kG, hi * hi);
        see(kPoly, largest(c[0], c[1], c[2], hi * hi));
        see(kPoly, largest(0.0, c[1], c[2], hi * hi));
        hi = std::max(1.01 * largest_step(c, hi), 1e-6);
        if (!(hi <= 8.0)) return false;
        x = std::max(x, hi);
    }
    if (pair && hyper.steps > 1) {
        // functions of one singular value, at most 1: by samples, as the factors' room is more than what lies between them
        constexpr int kSamples = 256;
        const double *c = hyper.coefficients[0], *e = hyper.coefficients[1];
        for (int i = 0; i <= kSamples; ++i) {
            const double s = 1.01 * i / kSamples, g = s * s, rest = c[1] * g + c[2] * g * g, poly = c[0] + rest;
            const double g2 = g * poly * poly, rest2 = e[1] * g2 + e[2] * g2 * g2;
            see(kR1, rest);
            see(kW, rest * g);
            see(kG2, g2);
            see(kR2, rest2);
            see(kQ, poly * (e[0] + rest2) - c[0] * e[0]);
        }
    }
    r->sigma = power_below(24000.0 / x);
    for (int i = 0; i < kRoles; ++i) {
        if (!(most[i] <= 16384.0)) return false;
        r->factor[i] = power_below(24000.0 / most[i]);
    }
    return true;
}

// The products of a step, in order: the first two iterations at once (a Gram matrix, five products of symmetric ones,
// one with X), where the handle makes them so, and single ones (Gram, polynomial, X).
constexpr int kPairPhases = 7;
int phase_kind(bool pair, int phase)
{
    if (pair && phase < kPairPhases) return phase == 0 ? kGram : phase == kPairPhases - 1 ? kNext : kSquare;
    const int k = (pair ? phase - kPairPhases : phase) % 3;
    return k == 0 ? kGram : k == 1 ? kSquare : kNext;
}
int phase_count(bool pair, int steps) { return pair ? kPairPhases + 3 * (steps - 2) : 3 * steps; }

// How tiles are cut: what a pair or block takes; the time of an inner block of it, what a tile costs besides, and the
// way from a product's end to the next one's first block.  Fitted to steps of three layers of a 256-wide network, four
// 512 wide, one 1024 and one 2048 wide, and eight matrices of mixed sizes, each cut all three ways (within 25 %, most
// 10): 256 x 256 tiles are best from 2048 on (1,120 us, 128 x 128 1,430), 128 x 128 at 512 (308; 340 and 365) and 1024
// (344; 385 and 410), 128 x 64 at 256 (105; 175 and 130).
struct Shape {
    int cg, bn;
    double block_us, tile_us, join_us;
};
constexpr Shape kShapes[] = {{2, 256, 0.40, 3.0, 8.0}, {1, 128, 0.22, 4.0, 3.0}, {1, 64, 0.19, 3.0, 3.0}};

// Of a symmetric product: the tiles with anything on or above the diagonal, in whole diagonal blocks.
bool kept(const Shape& S, int64_t a, int64_t b) { return b * S.bn >= a * 128 * S.cg; }
int64_t tile_rows(const Shape& S, int64_t rows) { return div_up(rows, 128 * S.cg); }
int64_t tile_cols(const Shape& S, int64_t cols) { return div_up(cols, S.bn); }
int64_t square_tiles(const Shape& S, int64_t m)
{
    int64_t n = 0;
    for (int64_t a = 0; a < tile_rows(S, m); ++a) n += tile_cols(S, m) - a * 128 * S.cg / S.bn;
    return n;
}

// Every product's tiles dealt to the workers (blocks, or pairs), each to the one that is free first once the product
// before is complete: as many whole steps as a call may ask for, since the list of fewer is its beginning.  Returns the
// time that five steps take; nothing is dealt where the work alone would take `limit`.  A tile's result does not depend
// on who makes it.
double deal_tiles(const zero_muon* h, const Shape& S, int64_t most_workers, double limit, std::vector<Piece>* out, std::vector<int32_t>* bounds)
{
    const size_t n = h->rows.size();
    std::vector<size_t> order;                // longest inner dimension first
    int64_t most = 0;
    for (size_t i = 0; i < n; ++i) {
        if (h->rows[i] * h->cols[i] == 0) continue;
        order.push_back(i);
        most += tile_rows(S, h->rows[i]) * tile_cols(S, h->cols[i]);
    }
    std::stable_sort(order.begin(), order.end(), [&](size_t a, size_t b) { return std::max(h->rows[a], h->cols[a]) > std::max(h->rows[b], h->cols[b]); });
    const int workers = (int)std::max<int64_t>(1, std::min(most_workers, most));
    const int phases = phase_count(h->pair, ZERO_MUON_MAX_STEPS), five = phase_count(h->pair, 5);
    double work = 0.0;
    for (const size_t i : order) {
        const int64_t r = h->rows[i], c = h->cols[i], m = std::min(r, c);
        const double whole = (double)(tile_rows(S, r) * tile_cols(S, c)), half = (double)square_tiles(S, m);
        for (int phase = 0; phase < five; ++phase) {
            const int kind = phase_kind(h->pair, phase);
            work += (kind == kNext ? whole : half) * ((double)div_up(kind == kGram ? std::max(r, c) : m, kBK) * S.block_us + S.tile_us);
        }
    }
    if (work / workers >= limit) return limit;
    std::vector<std::vector<Piece>> mine((size_t)workers);
    using Free = std::pair<double, int>;
    std::vector<Free> heap;
    for (int w = 0; w < workers; ++w) heap.push_back(Free(0.0, w));
    std::vector<double> complete(n, 0.0);
    double at_five = 0.0, end = 0.0;
    for (int phase = 0; phase < phases; ++phase) {
        const int kind = phase_kind(h->pair, phase);
        for (const size_t i : order) {
            const int64_t r = h->rows[i], c = h->cols[i], m = std::min(r, c), inner = kind == kGram ? std::max(r, c) : m;
            const int64_t tm = tile_rows(S, kind == kNext ? r : m), tn = tile_cols(S, kind == kNext ? c : m);
            const double each = div_up(inner, kBK) * S.block_us + S.tile_us;
            double last = 0.0;
            // groups of eight tile rows, column by column, so that what runs at one time shares its operands
            for (int64_t g = 0; g < tm; g += 8)
                for (int64_t b = 0; b < tn; ++b)
                    for (int64_t a = g; a < std::min(tm, g + 8); ++a) {
                        if (kind != kNext && !kept(S, a, b)) continue;
                        std::pop_heap(heap.begin(), heap.end(), std::greater<Free>());
                        Free& f = heap.back();
                        f.first = std::max(f.first, complete[i]) + each;
                        last = std::max(last, f.first);
                        mine[(size_t)f.second].push_back(Piece{(int32_t)((int64_t)i | (int64_t)phase << 16), (int32_t)(a << 16 | b)});
                        std::push_heap(heap.begin(), heap.end(), std::greater<Free>());
                    }
            complete[i] = last + S.join_us;
            end = std::max(end, complete[i]);
        }
        if (phase == five - 1) at_five = end;
    }
    out->clear();
    bounds->assign((size_t)workers * kMaxPhases, 0);
    for (int w = 0; w < workers; ++w) {
        int32_t* b = bounds->data() + (size_t)w * kMaxPhases;
        size_t k = 0;
        for (int phase = 0; phase < kMaxPhases; ++phase) {
            while (k < mine[(size_t)w].size() && (mine[(size_t)w][k].tensor >> 16) < phase) ++k;
            b[phase] = (int32_t)(out->size() + k);
        }
        out->insert(out->end(), mine[(size_t)w].begin(), mine[(size_t)w].end());
    }
    return at_five;
}

zero_status_t check_hyper(const zero_muon* h, const zero_muon_hyper_t* hyper, Range* range, const char* who)
{
    const std::string w = std::string(who) + ": ";
    if (!hyper) return fail(ZERO_EINVAL, w + "NULL argument");
    if (!(hyper->momentum >= 0.0 && hyper->momentum < 1.0)) return fail(ZERO_EINVAL, w + "momentum must be in [0, 1)");
    if (!std::isfinite(hyper->lr) || !std::isfinite(hyper->weight_decay) || !(hyper->eps >= 1e-12) || !std::isfinite(hyper->eps))
        return fail(ZERO_EINVAL, w + "bad hyperparameter");
    if (hyper->steps < 1 || hyper->steps > ZERO_MUON_MAX_STEPS) return fail(ZERO_EINVAL, w + "steps must be in 1 .. ZERO_MUON_MAX_STEPS");
    if (hyper->scale < ZERO_MUON_SCALE_NONE || hyper->scale > ZERO_MUON_SCALE_RMS) return fail(ZERO_EINVAL, w + "bad scale");
    if (hyper->flags & ~(int64_t)ZERO_MUON_NESTEROV) return fail(ZERO_EINVAL, w + "unknown flag");
    for (int k = 0; k < hyper->steps; ++k)
        for (int j = 0; j < 3; ++j)
            if (!std::isfinite(hyper->coefficients[k][j])) return fail(ZERO_EINVAL, w + "a coefficient is not finite");
    if (!find_range(*hyper, h && h->pair, range)) return fail(ZERO_ERANGE, w + "the coefficients let singular values of at most 1 grow beyond 8, or a polynomial of them beyond 16384");
    return ZERO_OK;
}

zero_status_t ready(const zero_muon* h, const char* who)
{
    if (!h) return fail(ZERO_EINVAL, std::string(who) + ": NULL handle");
    if (!h->bound) return fail(ZERO_ESTATE, std::string(who) + ": nothing bound (zero_muon_bind)");
    int dev = -1;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, who);
    if (dev != h->device) return fail(ZERO_EINVAL, std::string(who) + ": the bound buffers live on another device");
    return ZERO_OK;
}

MuonParams params(const zero_muon* h, const zero_muon_hyper_t& hyper, double loss_scale, const Range& range)
{
    char* ws = static_cast<char*>(h->workspace);
    MuonParams P;
    std::memset(&P, 0, sizeof(P));
    P.tensors = reinterpret_cast<MuonTensor*>(ws + h->at_tensors);
    P.grads = reinterpret_cast<const void* const*>(ws + h->at_grads);
    P.momentum[0] = h->momentum[0];
    P.momentum[1] = h->momentum[1];
    P.st = reinterpret_cast<MuonState*>(ws);
    P.slots = reinterpret_cast<double*>(ws + h->at_slots);
    P.scale = reinterpret_cast<float*>(ws + h->at_scale);
    P.tickets = reinterpret_cast<uint32_t*>(ws + h->at_tickets);
    P.counters = reinterpret_cast<uint32_t*>(ws + h->at_counters);
    P.n_counters = (int32_t)h->rows.size() * kMaxPhases;
    P.n_d = h->n_d;
    P.nesterov = (hyper.flags & ZERO_MUON_NESTEROV) != 0;
    P.inv = (float)(1.0 / ((double)h->n_d * loss_scale));
    P.mu = (float)hyper.momentum;
    P.nu = (float)(1.0 - hyper.momentum);
    P.sigma = (float)range.sigma;
    P.eps = hyper.eps;
    return P;
}

int pass_grid(int64_t pieces, int per_sm) { return (int)std::max<int64_t>(1, std::min<int64_t>(pieces, per_sm * kGb300Sms)); }

zero_status_t launch_reduce(const zero_muon* h, MuonParams P, cudaStream_t s)
{
    if (h->chunks.empty()) return ZERO_OK;
    P.pieces = reinterpret_cast<const Piece*>(static_cast<char*>(h->workspace) + h->at_chunks);
    P.count = (int32_t)h->chunks.size();
    const cudaError_t e = h->dtype16 == ZERO_BF16 ? launch_after(muon_reduce_kernel<ZERO_BF16>, pass_grid(P.count, kReduceBlocks), kThreads, 0, s, P)
                                                  : launch_after(muon_reduce_kernel<ZERO_FP16>, pass_grid(P.count, kReduceBlocks), kThreads, 0, s, P);
    return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "zero_muon: launch");
}

template <int CG, int BN>
zero_status_t launch_products(const zero_muon* h, const ProductParams& P, cudaStream_t s)
{
    constexpr int kShared = Tiles<CG, BN>::kScoutSmem;
    const cudaError_t set = allow_shared<muon_product_kernel<CG, BN>>(kShared);
    if (set != cudaSuccess) return cuda_fail(set, "zero_muon: shared memory");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(CG * h->running));
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = kShared;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeCooperative;
    attr.val.cooperative = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, muon_product_kernel<CG, BN>, P);
    return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "zero_muon: launch");
}

// Workers of the products that the current device has room for at one time: a cooperative launch of more is refused.
template <int CG, int BN>
cudaError_t resident_workers(int* workers)
{
    constexpr int kShared = Tiles<CG, BN>::kScoutSmem;
    cudaError_t e = allow_shared<muon_product_kernel<CG, BN>>(kShared);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)CG);
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = kShared;
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(workers, muon_product_kernel<CG, BN>, &cfg);
    return e;
}

// The first X, the iterations and the parameters.
zero_status_t launch_rest(const zero_muon* h, MuonParams P, const zero_muon_hyper_t& hyper, const Range& R, cudaStream_t s)
{
    P.pieces = reinterpret_cast<const Piece*>(static_cast<char*>(h->workspace) + h->at_groups);
    P.count = (int32_t)h->groups.size();
    const int grid = pass_grid(P.count, kStartBlocks);
    cudaError_t e = cudaSuccess;
    if (P.count > 0) {
        e = launch_after(muon_start_kernel, grid, kThreads, 0, s, P);
        if (e != cudaSuccess) return cuda_fail(e, "zero_muon: launch");
        char* ws = static_cast<char*>(h->workspace);
        ProductParams Q;
        std::memset(&Q, 0, sizeof(Q));
        Q.tensors = P.tensors;
        Q.tiles = reinterpret_cast<const Piece*>(ws + h->at_tiles);
        Q.bounds = reinterpret_cast<const int32_t*>(ws + h->at_bounds);
        Q.counters = P.counters;
        Q.st = P.st;
        Q.plan = P.plan;
        Q.how = hyper.scale;
        Q.bf = h->dtype16 == ZERO_BF16;
        Q.lr = (float)hyper.lr;
        Q.decay = (float)(hyper.lr * hyper.weight_decay);
        Q.wait_ns = (uint64_t)h->wait_ns;
        // one step alone of a handle that makes two at once is the first of the single ones
        const bool pair = h->pair && hyper.steps >= 2;
        Q.first = h->pair && !pair ? kPairPhases : 0;
        Q.last = Q.first + phase_count(pair, hyper.steps);
        int ops = 0, src = 0;
        auto op = [&](int kind) -> Op& {
            Op& o = Q.ops[ops++];
            o.kind = kind;
            o.src = src;
            return o;
        };
        // one symmetric product: out = f left right + l0 add0 + l1 add1 + d I, of values (their factors in fp16 are
        // range's)
        auto square = [&](Role left, Role right, Role out, double f, double d, std::initializer_list<std::pair<Role, double>> adds) {
            Op& o = op(kSquare);
            o.left = kSlot[left];
            o.right = kSlot[right];
            o.out = kSlot[out];
            o.scale = (float)(f * R.of(out) / (R.of(left) * R.of(right)));
            o.diag = (float)(d * R.of(out));
            for (const auto& a : adds) {
                o.add[o.adds] = kSlot[a.first];
                o.lin[o.adds++] = (float)(a.second * R.of(out) / R.of(a.first));
            }
        };
        auto gram = [&]() {
            Op& o = op(kGram);
            o.out = kSlot[kG];
            o.scale = (float)(R.of(kG) / (R.sigma * R.sigma));
        };
        // X <- poly X (+ d X where the polynomial is without d I, X with its low part)
        auto next = [&](Role poly, double d, bool keep_low) {
            Op& o = op(kNext);
            o.left = kSlot[poly];
            o.scale = (float)(1.0 / R.of(poly));
            if (d != 0.0) {
                o.adds = 2;
                o.lin[0] = (float)d;
                o.lin[1] = (float)(d / kLow);
            }
            o.keep_low = keep_low;
            src ^= 1;
        };
        int k = 0;
        if (pair) {
            // Two iterations at once.  The second's G is (a I + R1) G (a I + R1), R1 = b G + c G^2, as polynomials of G
            // commute: products of the smaller side instead of two passes over X, and nothing rounds the X between.
            const double *c = hyper.coefficients[0], *e = hyper.coefficients[1];
            gram();
            square(kG, kG, kR1, c[2], 0.0, {{kG, c[1]}});
            square(kR1, kG, kW, 1.0, 0.0, {});
            square(kR1, kW, kG2, 1.0, 0.0, {{kG, c[0] * c[0]}, {kW, 2.0 * c[0]}});
            square(kG2, kG2, kR2, e[2], 0.0, {{kG2, e[1]}});
            square(kR2, kR1, kQ, 1.0, 0.0, {{kR1, e[0]}, {kR2, c[0]}});
            next(kQ, c[0] * e[0], false);
            k = 2;
        }
        for (; k < hyper.steps; ++k) {
            const double* c = hyper.coefficients[k];
            const bool twice = !pair && k < kTwice;
            gram();
            square(kG, kG, kPoly, c[2], twice ? 0.0 : c[0], {{kG, c[1]}});
            next(kPoly, twice ? c[0] : 0.0, twice && k + 1 < kTwice && k + 1 < hyper.steps);
        }
        Op& end = Q.ops[ops - 1];
        end.final = 1;
        end.scale /= (float)R.sigma;
        end.lin[0] /= (float)R.sigma;
        end.lin[1] /= (float)R.sigma;
        return h->cg == 2 ? launch_products<2, 256>(h, Q, s) : h->bn == 128 ? launch_products<1, 128>(h, Q, s) : launch_products<1, 64>(h, Q, s);
    }
    e = launch_after(muon_close_kernel, 1, 32, 0, s, P.st, P.plan);
    return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "zero_muon: launch");
}

zero_status_t plan_ready(const zero_muon* h, const zero_plan* plan, const char* who)
{
    if (!h || !plan) return fail(ZERO_EINVAL, std::string(who) + ": NULL argument");
    const zero_status_t st = ready(h, who);
    if (st != ZERO_OK) return st;
    if (!plan->workspace) return fail(ZERO_ESTATE, std::string(who) + ": no rank of the plan is bound");
    if (plan->device != h->device) return fail(ZERO_EINVAL, std::string(who) + ": the plan lives on another device");
    return ZERO_OK;
}

// Elements of X, and of G, in the workspace: each buffer starts on 256 bytes.
int64_t x_elems(int64_t rows, int64_t cols) { return up(rows * up(cols, kRowElems), 128); }
int64_t g_elems(int64_t m) { return up(m * up(m, kRowElems), 128); }

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" {

zero_status_t zero_muon_create(const int64_t* rows, const int64_t* cols, int64_t n_matrices, int n_contribs, int dtype16, zero_muon_t** out)
try {
    if (!out || ((!rows || !cols) && n_matrices > 0)) return fail(ZERO_EINVAL, "zero_muon_create: NULL argument");
    *out = nullptr;
    if (n_matrices < 0) return fail(ZERO_EINVAL, "zero_muon_create: negative count");
    if (n_matrices > ZERO_MUON_MAX_MATRICES) return fail(ZERO_ERANGE, "zero_muon_create: more than ZERO_MUON_MAX_MATRICES matrices");
    if (n_contribs < 1) return fail(ZERO_EINVAL, "zero_muon_create: n_contribs must be at least 1");
    if (n_contribs > ZERO_MAX_RANKS) return fail(ZERO_ERANGE, "zero_muon_create: more than ZERO_MAX_RANKS contributions");
    if (dtype16 != ZERO_BF16 && dtype16 != ZERO_FP16) return fail(ZERO_EINVAL, "zero_muon_create: bad dtype16");
    std::unique_ptr<zero_muon> h(new zero_muon);
    h->n_d = n_contribs;
    h->dtype16 = dtype16;
    int64_t at = 0;
    for (int64_t i = 0; i < n_matrices; ++i) {
        const int64_t r = rows[i], c = cols[i];
        if (r < 0 || c < 0) return fail(ZERO_EINVAL, "zero_muon_create: negative size");
        if (r > ZERO_MUON_MAX_SIZE || c > ZERO_MUON_MAX_SIZE || std::min(r, c) > ZERO_MUON_MAX_SIDE)
            return fail(ZERO_ERANGE, "zero_muon_create: a matrix beyond ZERO_MUON_MAX_SIZE, or its smaller side beyond ZERO_MUON_MAX_SIDE");
        h->elems += r * c;
        if (h->elems > (int64_t)1 << 40) return fail(ZERO_ERANGE, "zero_muon_create: more than 2^40 elements");   // pieces stay 32-bit
        h->state_elems += up(r * c, kStateBlock);
    }
    h->rows.assign(rows, rows + n_matrices);
    h->cols.assign(cols, cols + n_matrices);
    for (int64_t i = 0; i < n_matrices; ++i) {
        const int64_t r = rows[i], c = cols[i];
        for (int64_t k = 0; k < div_up(r * c, kChunk); ++k) h->chunks.push_back(Piece{(int32_t)i, (int32_t)k});
        for (int64_t k = 0; k < div_up(r * up(c, kRowElems), kChunk); ++k) h->groups.push_back(Piece{(int32_t)i, (int32_t)k});
    }
    // Two iterations at once replace two passes over X by products of the smaller side, and are as exact from sides of
    // 64 on; for small sides the second G's largest values, differences of larger terms, are not.
    h->pair = h->elems > 0;
    for (int64_t i = 0; i < n_matrices; ++i)
        if (rows[i] * cols[i] > 0 && std::min(rows[i], cols[i]) < kPairSide) h->pair = false;
    if (h->elems > 0) {
        double best = 1e30;
        for (const Shape& S : kShapes) {
            std::vector<Piece> tiles;
            std::vector<int32_t> bounds;
            const double us = deal_tiles(h.get(), S, kGb300Sms / S.cg, best, &tiles, &bounds);
            if (us >= best) continue;
            best = us;
            h->cg = S.cg;
            h->bn = S.bn;
            h->tiles.swap(tiles);
            h->bounds.swap(bounds);
        }
        if (h->tiles.size() > (size_t)INT32_MAX) return fail(ZERO_ERANGE, "zero_muon_create: too many tiles");
        h->workers = (int)(h->bounds.size() / kMaxPhases);
    }
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += up(bytes, 256);
        return here;
    };
    take(sizeof(MuonState));
    h->at_tensors = take((int64_t)sizeof(MuonTensor) * n_matrices);
    h->at_grads = take(8 * n_matrices * n_contribs);
    h->at_chunks = take(8 * (int64_t)h->chunks.size());
    h->at_groups = take(8 * (int64_t)h->groups.size());
    h->at_tiles = take(8 * (int64_t)h->tiles.size());
    h->at_bounds = take(4 * (int64_t)h->bounds.size());
    h->at_counters = take(4 * n_matrices * kMaxPhases);
    h->at_slots = take(8 * (int64_t)h->chunks.size());
    h->at_scale = take(4 * n_matrices);
    h->at_tickets = take(4 * n_matrices);
    h->at_data = at;
    for (int64_t i = 0; i < n_matrices; ++i)
        if (rows[i] * cols[i] > 0) at += 2 * (3 * x_elems(rows[i], cols[i]) + kSquares * g_elems(std::min(rows[i], cols[i])));
    h->bytes = at;
    *out = h.release();
    return ZERO_OK;
}
catch (...) {
    return exception_status("zero_muon_create");
}

zero_status_t zero_muon_info(const zero_muon_t* h, zero_muon_info_t* out)
try {
    if (!h || !out) return fail(ZERO_EINVAL, "zero_muon_info: NULL argument");
    out->n_matrices = (int64_t)h->rows.size();
    out->n_contribs = h->n_d;
    out->elems = h->elems;
    out->state_elems = h->state_elems;
    out->workspace_bytes = h->bytes;
    return ZERO_OK;
}
catch (...) {
    return exception_status("zero_muon_info");
}

zero_status_t zero_muon_set_option(zero_muon_t* h, int option, int64_t value)
try {
    if (!h) return fail(ZERO_EINVAL, "zero_muon_set_option: NULL handle");
    switch (option) {
    case ZERO_MUON_OPT_WAIT_LIMIT_NS:
        if (value < 0 || value > ZERO_MUON_MAX_WAIT_NS) return fail(ZERO_EINVAL, "zero_muon_set_option: the wait limit must be in 0 .. ZERO_MUON_MAX_WAIT_NS");
        h->wait_ns = value;
        return ZERO_OK;
    case ZERO_MUON_OPT_SMS:
        if (value < 0 || value == 1) return fail(ZERO_EINVAL, "zero_muon_set_option: SMs must be 0 (all) or at least 2");
        h->most_sms = value;
        return ZERO_OK;
    default: return fail(ZERO_EINVAL, "zero_muon_set_option: unknown option");
    }
}
catch (...) {
    return exception_status("zero_muon_set_option");
}

zero_status_t zero_muon_bind(zero_muon_t* h, float* const* params, void* const* params16, void* const* updates, const void* const* grads,
                             float* const momentum[2], void* workspace, int64_t t, void* stream)
try {
    if (!h) return fail(ZERO_EINVAL, "zero_muon_bind: NULL handle");
    const size_t n = h->rows.size();
    if (n > 0 && !grads) return fail(ZERO_EINVAL, "zero_muon_bind: NULL argument");
    if (!workspace) return fail(ZERO_EINVAL, "zero_muon_bind: workspace is NULL");
    if (!aligned(workspace, 256)) return fail(ZERO_EALIGN, "zero_muon_bind: workspace not 256-byte aligned");
    if (t < -1 || (t == -1 && (!h->bound || workspace != h->workspace)))
        return fail(ZERO_EINVAL, "zero_muon_bind: t must be >= 0 (-1 keeps an earlier bind's, with its workspace)");
    if (h->state_elems > 0) {
        if (!momentum || !momentum[0] || !momentum[1]) return fail(ZERO_EINVAL, "zero_muon_bind: NULL momentum");
        if (momentum[0] == momentum[1]) return fail(ZERO_EINVAL, "zero_muon_bind: the momentum's halves are one buffer");
        if (!aligned(momentum[0], 16) || !aligned(momentum[1], 16)) return fail(ZERO_EALIGN, "zero_muon_bind: momentum not 16-byte aligned");
        if (t == -1 && (momentum[0] != h->momentum[0] || momentum[1] != h->momentum[1]))
            return fail(ZERO_EINVAL, "zero_muon_bind: t = -1 keeps the momentum too");
    }
    char* ws = static_cast<char*>(workspace);
    std::vector<unsigned char> image((size_t)h->at_data, 0);
    MuonState init;
    std::memset(&init, 0, sizeof(init));
    init.t = t;
    std::memcpy(image.data(), &init, sizeof(init));
    const void** table = reinterpret_cast<const void**>(image.data() + h->at_grads);
    int64_t data = h->at_data, at = 0;
    for (size_t i = 0; i < n; ++i) {
        const int64_t r = h->rows[i], c = h->cols[i], m = std::min(r, c);
        MuonTensor T;
        std::memset(&T, 0, sizeof(T));
        T.rows = (int32_t)r;
        T.cols = (int32_t)c;
        T.m = (int32_t)m;
        if (m > 0) {
            T.ldx = (int32_t)up(c, kRowElems);
            T.ldm = (int32_t)up(m, kRowElems);
            T.wide = r <= c;
            T.at = at;
            const Shape cut{h->cg, h->bn, 0.0, 0.0, 0.0};
            T.tiles[0] = (int32_t)square_tiles(cut, m);
            T.tiles[1] = (int32_t)(tile_rows(cut, r) * tile_cols(cut, c));
            T.chunks = (int32_t)div_up(r * c, kChunk);
            T.aspect = (float)std::sqrt(std::max(1.0, (double)r / (double)c));
            T.rms = (float)(0.2 * std::sqrt((double)std::max(r, c)));
            T.p = params ? params[i] : nullptr;
            T.p16 = params16 ? static_cast<uint16_t*>(params16[i]) : nullptr;
            T.update = updates ? static_cast<uint16_t*>(updates[i]) : nullptr;
            if (!T.p && T.p16) return fail(ZERO_EINVAL, "zero_muon_bind: a 16-bit copy without its parameters");
            if (!T.p && !T.update) return fail(ZERO_EINVAL, "zero_muon_bind: a matrix with neither parameters nor update");
            if (!aligned(T.p, 4) || !aligned(T.p16, 2) || !aligned(T.update, 2))
                return fail(ZERO_EALIGN, "zero_muon_bind: a matrix is not aligned to its element size");
            T.vec_g = 1;
            for (int k = 0; k < h->n_d; ++k) {
                const void* g = grads[(size_t)k * n + i];
                if (!g) return fail(ZERO_EINVAL, "zero_muon_bind: NULL contribution");
                if (!aligned(g, 2)) return fail(ZERO_EALIGN, "zero_muon_bind: a contribution is not aligned to 2 bytes");
                T.vec_g = T.vec_g && aligned(g, 16);
                table[i * (size_t)h->n_d + (size_t)k] = g;
            }
            T.vec_p = c % 4 == 0 && aligned(T.p, 16) && aligned(T.p16, 8) && aligned(T.update, 8);
            uint16_t* q = reinterpret_cast<uint16_t*>(ws + data);
            const int64_t x = x_elems(r, c), g = g_elems(m);
            T.x[0] = q;
            T.x[1] = q + x;
            T.low = q + 2 * x;
            for (int k = 0; k < kSquares; ++k) T.square[k] = q + 3 * x + k * g;
            data += 2 * (3 * x + kSquares * g);
            zero_status_t st = ZERO_OK;
            auto map = [&](int which, const Operand& o) {
                if (st == ZERO_OK) st = encode(&T.map[which], o, ZERO_FP16, box_rows(h->bn), "zero_muon_bind");
            };
            auto out = [&](int which, const void* p, int64_t rows, int64_t cols, int64_t ld) {
                if (st == ZERO_OK) st = encode_box(&T.map[which], p, rows, cols, ld, ZERO_FP16, 32, 32, "zero_muon_bind");
            };
            for (int k = 0; k < 2; ++k) {
                map(kMapX + k, Operand{T.x[k], r, c, T.ldx, false});
                map(kMapXAcross + k, Operand{T.x[k], c, r, T.ldx, true});
                out(kMapOutX + k, T.x[k], r, c, T.ldx);
            }
            out(kMapOutLow, T.low, r, c, T.ldx);
            for (int k = 0; k < kSquares; ++k) {
                map(kMapSquare + k, Operand{T.square[k], m, m, T.ldm, false});
                map(kMapSquareAcross + k, Operand{T.square[k], m, m, T.ldm, true});
                out(kMapOutSquare + k, T.square[k], m, m, T.ldm);
            }
            if (st != ZERO_OK) return st;
            at += up(r * c, kStateBlock);
        }
        std::memcpy(image.data() + h->at_tensors + (int64_t)sizeof(T) * (int64_t)i, &T, sizeof(T));
    }
    auto put = [&](int64_t where, const std::vector<Piece>& v) {
        if (!v.empty()) std::memcpy(image.data() + where, v.data(), v.size() * sizeof(Piece));
    };
    put(h->at_chunks, h->chunks);
    put(h->at_groups, h->groups);
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "zero_muon_bind: cudaGetDevice");
    int running = h->workers;
    if (running > 0) {
        int resident = 0;
        e = h->cg == 2 ? resident_workers<2, 256>(&resident) : h->bn == 128 ? resident_workers<1, 128>(&resident) : resident_workers<1, 64>(&resident);
        if (e != cudaSuccess) return cuda_fail(e, "zero_muon_bind: the blocks that the device has room for");
        if (resident < 1) return fail(ZERO_ECUDA, "zero_muon_bind: the device has no room for a block of the products");
        running = std::min(running, resident);
        if (h->most_sms > 0) running = std::min(running, (int)std::max<int64_t>(1, std::min<int64_t>(h->most_sms, kGb300Sms) / h->cg));
    }
    std::vector<Piece> fewer_tiles;
    std::vector<int32_t> fewer_bounds;
    const bool fewer = running < h->workers;
    if (fewer) {
        // the same tiles among the workers that there are
        for (const Shape& S : kShapes)
            if (S.cg == h->cg && S.bn == h->bn) deal_tiles(h, S, running, 1e30, &fewer_tiles, &fewer_bounds);
    }
    put(h->at_tiles, fewer ? fewer_tiles : h->tiles);
    const std::vector<int32_t>& bounds = fewer ? fewer_bounds : h->bounds;
    if (!bounds.empty()) std::memcpy(image.data() + h->at_bounds, bounds.data(), bounds.size() * sizeof(int32_t));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t skip = t == -1 ? 256 : 0;       // -1: the state's slot stays
    e = cudaMemcpyAsync(ws + skip, image.data() + skip, image.size() - skip, cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e, "zero_muon_bind: the workspace's tables");
    for (int k = 0; k < 2; ++k) h->momentum[k] = momentum ? momentum[k] : nullptr;
    h->workspace = workspace;
    h->checked_in = 0;                           // what a check left there is gone
    h->device = dev;
    h->running = running;
    h->bound = true;
    return ZERO_OK;
}
catch (...) {
    return exception_status("zero_muon_bind");
}

zero_status_t zero_muon_step(zero_muon_t* h, const zero_muon_hyper_t* hyper, double loss_scale, void* stream)
try {
    if (!h) return fail(ZERO_EINVAL, "zero_muon_step: NULL handle");
    Range R;
    zero_status_t st = check_hyper(h, hyper, &R, "zero_muon_step");
    if (st != ZERO_OK) return st;
    if (!(loss_scale > 0.0) || !std::isfinite(loss_scale)) return fail(ZERO_EINVAL, "zero_muon_step: loss_scale must be positive");
    st = ready(h, "zero_muon_step");
    if (st != ZERO_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const MuonParams P = params(h, *hyper, loss_scale, R);
    h->checked_in = 0;                           // the other half of the momentum is this step's now
    st = launch_reduce(h, P, s);
    return st == ZERO_OK ? launch_rest(h, P, *hyper, R, s) : st;
}
catch (...) {
    return exception_status("zero_muon_step");
}

zero_status_t zero_muon_check(zero_muon_t* h, zero_plan_t* plan, const zero_muon_hyper_t* hyper, void* stream)
try {
    Range R;
    zero_status_t st = check_hyper(h, hyper, &R, "zero_muon_check");
    if (st == ZERO_OK) st = plan_ready(h, plan, "zero_muon_check");
    if (st != ZERO_OK) return st;
    if (h->checked_in == plan->step_no) return fail(ZERO_ESTATE, "zero_muon_check: already part of this step");
    if (plan->in_step && plan->offload)
        return fail(ZERO_ESTATE, "zero_muon_check: must precede the first bucket/unit of a step that is offloaded");
    if (plan->moved_in == plan->step_no) return fail(ZERO_ESTATE, "zero_muon_check: a part of this step, which it could not leave out, is enqueued");
    MuonParams P = params(h, *hyper, 1.0, R);
    P.plan = reinterpret_cast<DevState*>(plan->workspace);
    st = launch_reduce(h, P, static_cast<cudaStream_t>(stream));
    if (st != ZERO_OK) return st;
    h->checked_in = plan->step_no;
    h->checked_mu = hyper->momentum;
    h->checked_flags = hyper->flags;
    return ZERO_OK;
}
catch (...) {
    return exception_status("zero_muon_check");
}

zero_status_t zero_muon_step_with(zero_muon_t* h, zero_plan_t* plan, const zero_muon_hyper_t* hyper, void* stream)
try {
    Range R;
    zero_status_t st = check_hyper(h, hyper, &R, "zero_muon_step_with");
    if (st == ZERO_OK) st = plan_ready(h, plan, "zero_muon_step_with");
    if (st != ZERO_OK) return st;
    if (h->checked_in != plan->step_no) return fail(ZERO_ESTATE, "zero_muon_step_with: needs zero_muon_check in the same step");
    if (h->stepped_in == plan->step_no) return fail(ZERO_ESTATE, "zero_muon_step_with: already part of this step");
    bool all = plan->in_step;
    for (int64_t b = 0; b < plan->n_buckets && all; ++b) all = plan->covered[(size_t)b] != 0;
    if (!all) return fail(ZERO_ESTATE, "zero_muon_step_with: follows the step of every bucket/unit, before the step's finish");
    if (hyper->momentum != h->checked_mu || hyper->flags != h->checked_flags)
        return fail(ZERO_EINVAL, "zero_muon_step_with: one step has one momentum and one set of flags");
    MuonParams P = params(h, *hyper, 1.0, R);
    P.plan = reinterpret_cast<DevState*>(plan->workspace);
    plan->moved_in = plan->step_no;
    st = launch_rest(h, P, *hyper, R, static_cast<cudaStream_t>(stream));
    if (st != ZERO_OK) return st;
    if (plan->offload) {
        // the host's update reads the step's state behind this event, and a wait that runs out here discards the step
        const cudaError_t e = cudaEventRecord((cudaEvent_t)plan->off_flag_event, static_cast<cudaStream_t>(stream));
        if (e != cudaSuccess) return cuda_fail(e, "zero_muon_step_with: event");
    }
    h->stepped_in = plan->step_no;
    return ZERO_OK;
}
catch (...) {
    return exception_status("zero_muon_step_with");
}

zero_status_t zero_muon_read(zero_muon_t* h, void* stream, zero_step_result_t* out)
try {
    if (!h || !out) return fail(ZERO_EINVAL, "zero_muon_read: NULL argument");
    const zero_status_t st = ready(h, "zero_muon_read");
    if (st != ZERO_OK) return st;
    MuonState state;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemcpyAsync(&state, h->workspace, sizeof(state), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e, "zero_muon_read");
    std::memset(out, 0, sizeof(*out));
    out->skipped = (int32_t)state.last_skipped;
    out->current = (int32_t)state.cur;
    out->t = state.t;
    out->scale = 1.0;
    out->good_steps = state.t;
    out->skipped_total = state.skipped;
    out->finished = state.finished;
    out->grad_norm = -1.0;
    if (state.timeout) {
        e = cudaMemsetAsync(&static_cast<MuonState*>(h->workspace)->timeout, 0, sizeof(state.timeout), s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
        if (e != cudaSuccess) return cuda_fail(e, "zero_muon_read: clearing the state");
        return fail(ZERO_ETIMEOUT, "zero_muon_read: a wait of a step's products ran out; its parameters may be partly moved, and the steps since then were left out");
    }
    return ZERO_OK;
}
catch (...) {
    return exception_status("zero_muon_read");
}

void zero_muon_destroy(zero_muon_t* h) { delete h; }

}  // extern "C"
