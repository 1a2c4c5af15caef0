// zero_norm.cu -- the norm after one block and the norm before the next, with the block's gate and
// residual scale, and their gradients (zero_block_norm_*):
//   u = Norm_post(h);  y = x + s gate u;  z = Norm_pre(y)
//
// A row is held in registers, from its only read to its only write: 8 bytes an element forward (h, x, y, z),
// 12 backward (h, y, dy, dz, dx, dh; the statistics are formed again from h and y, which are read
// anyway).  HBM would bound it; what does is issue: about 30 instructions an element forward, 57
// backward, half of them widening 16-bit values and moving them into pairs.  So all arithmetic is on
// pairs (one instruction for two fp32 operations), a thread holds as many elements as its registers
// allow, so that a row's sums and addresses are shared by more, and rows come through shared memory.
// Measured on one GB300: 16384 x 2048, LayerNorm with a gate, 52 us (5.2 TB/s, 0.76 of the copy rate);
// gradients of 16384 x 4096, RMS with gates, 188.7 us (4.3 TB/s, 0.63), of which 8 are the second kernel's;
// of 1001 x 1023, LayerNorm, gates of 7 rows, element by element, 23.7 us.
//
// Backward, per row (Layer centres h and y; RMS does not):
//   g = dz w_pre;   dx = dy + r_y (g - mean(g) - yn mean(g yn)),   yn the normalised y
//   du = s gate dx; d = du w_post;  dh = r_h (d - mean(d) - hn mean(d hn))
//   dw_pre = sum dz yn, db_pre = sum dz, dw_post = sum du hn, db_post = sum du, dgate = sum s dx u
// The last five are summed over rows: a worker (one block, or one warp for short rows) takes
// consecutive rows and keeps its sums in registers (in shared memory for rows beyond 4096
// elements, whose threads have too few registers); a second kernel adds the workers' sums in order.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "zero_device.cuh"

namespace zero {
namespace {

// A norm's weights.  Where there are none the pointer is to eight ones (or zeros) and the mask takes
// every element to them: no branch, no selection.
struct Weights {
    const uint16_t* p;
    uint32_t mask;
};
__device__ __align__(16) uint16_t g_no_weights[3][8] = {{0x3F80, 0x3F80, 0x3F80, 0x3F80, 0x3F80, 0x3F80, 0x3F80, 0x3F80},
                                                        {0x3C00, 0x3C00, 0x3C00, 0x3C00, 0x3C00, 0x3C00, 0x3C00, 0x3C00},
                                                        {0, 0, 0, 0, 0, 0, 0, 0}};   // ones in bf16, in fp16; zeros

struct NormParams {
    const uint16_t *h, *x, *gate, *dy, *dz;
    Weights post_w, post_b, pre_w, pre_b;
    const uint16_t* y_in;
    uint16_t *y, *z, *dx, *dh, *dgate;
    int64_t rows, ld_h, ld_x, ld_y, ld_z, ld_gate, ld_dy, ld_dz, ld_dx, ld_dh, ld_dgate;
    int64_t gate_rows;         // rows that share a gate row
    float* sums;               // [worker][4][dim]: dpre_w, dpre_b, dpost_w, dpost_b
    float* gate_sums;          // [worker][2][dim]: a gate group's part in the worker's first / last rows
    int64_t chunk;             // backward: consecutive rows a worker takes
    int32_t dim, post, pre;
    int32_t bias_sums;         // the biases' gradients are asked for
    float eps, scale, inv_dim;
};

// How rows are accessed: every row starts on 16 bytes and all threads hold as much (kEven), or some hold
// less (kRagged); or elements come one by one (kScalar).
enum { kEven = 0, kRagged = 1, kScalar = 2 };

// Which elements of a row a thread holds: V times eight.  Where every row starts on 16 bytes eight
// neighbours, else every T-th, so that a warp's accesses are to neighbouring elements either way.
template <int MODE, int V>
struct Lane {
    int tid, T, n;             // n: elements held (VEC: eights)
    __device__ __forceinline__ Lane(int tid_, int T_, int dim) : tid(tid_), T(T_)
    {
        if constexpr (MODE == kEven) n = V;
        else if constexpr (MODE == kRagged) n = tid * 8 < dim ? (dim - tid * 8 + 8 * T - 1) / (8 * T) : 0;
        else n = tid < dim ? (dim - tid + T - 1) / T : 0;
    }
    __device__ __forceinline__ int at(int k) const { return MODE != kScalar ? ((k >> 3) * T + tid) * 8 + (k & 7) : tid + k * T; }
};

// V times eight 16-bit elements as loaded.
template <int V>
struct Raw {
    uint32_t w[4 * V];
};

template <int MODE, int V>
__device__ __forceinline__ Raw<V> load_raw(const uint16_t* p, const Lane<MODE, V>& L)
{
    Raw<V> r;
    if constexpr (MODE != kScalar) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            uint4 q;
            if (MODE == kEven || v < L.n) q = *reinterpret_cast<const uint4*>(p + (v * L.T + L.tid) * 8);
            else q = make_uint4(0u, 0u, 0u, 0u);
            r.w[4 * v] = q.x; r.w[4 * v + 1] = q.y; r.w[4 * v + 2] = q.z; r.w[4 * v + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4 * V; ++k) {
            const uint32_t lo = 2 * k < L.n ? p[L.at(2 * k)] : 0u, hi = 2 * k + 1 < L.n ? p[L.at(2 * k + 1)] : 0u;
            r.w[k] = lo | (hi << 16);
        }
    }
    return r;
}

template <int DT>
__device__ __forceinline__ F2 widen(uint32_t w)
{
    float a, b;
    widen2<DT>(w, a, b);
    return pair(a, b);
}

// Plain loads: the kernel just before may be the one that writes the weights, and has not ended when this one
// is launched, so that they are not constant for its lifetime (what __ldg asks for).
template <int MODE, int V>
__device__ __forceinline__ Raw<V> load_weight(const Weights& W, const Lane<MODE, V>& L)
{
    Raw<V> r;
    if constexpr (MODE != kScalar) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            uint4 q;
            if (MODE == kEven || v < L.n) q = *reinterpret_cast<const uint4*>(W.p + (((v * L.T + L.tid) * 8) & W.mask));
            else q = make_uint4(0u, 0u, 0u, 0u);
            r.w[4 * v] = q.x; r.w[4 * v + 1] = q.y; r.w[4 * v + 2] = q.z; r.w[4 * v + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4 * V; ++k) {
            const uint32_t lo = 2 * k < L.n ? W.p[L.at(2 * k) & W.mask] : 0u, hi = 2 * k + 1 < L.n ? W.p[L.at(2 * k + 1) & W.mask] : 0u;
            r.w[k] = lo | (hi << 16);
        }
    }
    return r;
}

template <int DT, int MODE, int V>
__device__ __forceinline__ void store_row(uint16_t* p, const Lane<MODE, V>& L, const F2 (&x)[4 * V])
{
#pragma unroll
    for (int v = 0; v < V; ++v) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float a, b;
            split(x[4 * v + k], a, b);
            w[k] = narrow2<DT>(a, b);
        }
        if constexpr (MODE != kScalar) {
            if (MODE == kEven || v < L.n) *reinterpret_cast<uint4*>(p + (v * L.T + L.tid) * 8) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (8 * v + k < L.n) p[L.at(8 * v + k)] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
        }
    }
}

// A worker's fp32 sums: dim floats, not aligned beyond 4 bytes where dim is odd.
template <int MODE, int V>
__device__ __forceinline__ void store_sums(float* p, const Lane<MODE, V>& L, const F2 (&x)[4 * V])
{
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float t[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) split(x[4 * v + k], t[2 * k], t[2 * k + 1]);
        if constexpr (MODE != kScalar) {
            if (MODE == kEven || v < L.n) {
                float4* q = reinterpret_cast<float4*>(p + (v * L.T + L.tid) * 8);
                q[0] = make_float4(t[0], t[1], t[2], t[3]);
                q[1] = make_float4(t[4], t[5], t[6], t[7]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (8 * v + k < L.n) p[L.at(8 * v + k)] = t[k];
        }
    }
}

__device__ __forceinline__ float total(F2 x)
{
    float a, b;
    split(x, a, b);
    return a + b;
}

// What a thread does not hold becomes 0.
template <int MODE, int V>
__device__ __forceinline__ void clear_rest(const Lane<MODE, V>& L, F2 (&x)[4 * V])
{
#pragma unroll
    for (int k = 0; k < 4 * V; ++k) {
        if constexpr (MODE != kScalar) {
            if ((k >> 2) >= L.n) x[k] = both(0.0f);
        } else {
            float a, b;
            split(x[k], a, b);
            x[k] = pair(2 * k < L.n ? a : 0.0f, 2 * k + 1 < L.n ? b : 0.0f);
        }
    }
}

// One pair of them: 0 where the thread does not hold it.
template <int MODE, int V>
__device__ __forceinline__ F2 held(const Lane<MODE, V>& L, int k, F2 x)
{
    if constexpr (MODE != kScalar) {
        return (k >> 2) < L.n ? x : both(0.0f);
    } else {
        float a, b;
        split(x, a, b);
        return pair(2 * k < L.n ? a : 0.0f, 2 * k + 1 < L.n ? b : 0.0f);
    }
}

// Sums of NV values over the T threads of a row, the same bits in every thread.  `turn` picks one
// of two areas, so that one barrier a sum is enough.
constexpr int kSumArea = 4 * 32;

// Two values summed over lanes whose numbers differ in bit `o`: a in the lanes without it, b in the others.
__device__ __forceinline__ float fold(float a, float b, int o, int lane)
{
    const bool up = lane & o;
    const float keep = up ? b : a, give = up ? a : b;
    return keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
}

template <int NV>
__device__ __forceinline__ void row_sum(float (&v)[NV], int T, float* area, int& turn)
{
    const int lane = threadIdx.x & 31;
    if (T <= 32) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
        return;
    }
    // within the warp: lane l ends with value l % 4's sum (l % 2's of two, of one the sum itself)
    float x;
    if constexpr (NV == 1) {
        x = v[0] + __shfl_xor_sync(0xFFFFFFFFu, v[0], 1);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 2);
    } else if constexpr (NV == 2) {
        x = fold(v[0], v[1], 1, lane);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 2);
    } else {
        x = fold(fold(v[0], v[1], 1, lane), fold(v[2], NV > 3 ? v[NV - 1] : 0.0f, 1, lane), 2, lane);
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    float* s = area + turn * kSumArea;
    turn ^= 1;
    const int warp = threadIdx.x >> 5, warps = T >> 5;
    if (lane < NV) s[lane * 32 + warp] = x;
    __syncthreads();
    if (warps <= 4) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const float4 q = *reinterpret_cast<const float4*>(s + k * 32);
            v[k] = q.x + q.y;
            if (warps > 2) v[k] += q.z;
            if (warps > 3) v[k] += q.w;
        }
        return;
    }
    // lane l: value l / 8, warps l % 8, and 8 and 16 and 24 on
    const int k = lane >> 3;
    x = 0.0f;
    if (k < NV)
        for (int w = lane & 7; w < warps; w += 8) x += s[k * 32 + w];
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, x, i * 8);
}

// x centred (LAYER) in place, and 1 / sqrt(mean square + eps).
template <bool LAYER, int MODE, int V>
__device__ __forceinline__ float centre(F2 (&x)[4 * V], const Lane<MODE, V>& L, const NormParams& P, int T, float* area, int& turn)
{
    float s[1];
    if constexpr (LAYER) {
        F2 sum = x[0];
#pragma unroll
        for (int k = 1; k < 4 * V; ++k) sum = add(sum, x[k]);
        s[0] = total(sum);
        row_sum(s, T, area, turn);
        const F2 minus_mean = both(-s[0] * P.inv_dim);
#pragma unroll
        for (int k = 0; k < 4 * V; ++k) x[k] = add(x[k], minus_mean);
        if constexpr (MODE != kEven) clear_rest<MODE, V>(L, x);
    }
    F2 sum = mul(x[0], x[0]);
#pragma unroll
    for (int k = 1; k < 4 * V; ++k) sum = fma(x[k], x[k], sum);
    s[0] = total(sum);
    row_sum(s, T, area, turn);
    return rsqrtf(s[0] * P.inv_dim + P.eps);
}

// The gate row of consecutive or strided rows, without a division a row.
struct GateRow {
    int64_t group, rest, step_group, step_rest, rows;
    __device__ __forceinline__ GateRow(int64_t row, int64_t step, int64_t rows_)
        : group(row / rows_), rest(row % rows_), step_group(step / rows_), step_rest(step % rows_), rows(rows_)
    {
    }
    __device__ __forceinline__ void next()
    {
        group += step_group;
        rest += step_rest;
        if (rest >= rows) {
            rest -= rows;
            ++group;
        }
    }
};

// ---------------------------------------------------------------- rows on their way
//
// Even rows of two warps and more come through shared memory: one thread
// issues a bulk copy a tensor (TMA) for the row STAGES - 1 ahead, all on one mbarrier of that row's
// stage, and no thread's registers wait for memory.  A stage is free again once every thread has passed
// the first sum of the next row.  Measured on GB300: forward (16384 x 2048, LayerNorm) two stages 57 us,
// three 55, registers instead 72; backward (16384 x 4096, RMS) two stages 194, three 230 (they leave
// the weights little L1), registers instead 320.  Waits are bounded; one that runs out is reported
// (zero_operators_check), is the last one that its thread makes, and leaves the control flow as it is.
constexpr int kForwardStages = 3, kBackwardStages = 2;
constexpr uint64_t kRowWaitNs = 1000000000ull;
__device__ uint32_t g_norm_error;

template <int STAGES>
struct RowPipe {
    uint32_t bars, data, stage_bytes, row_bytes;
    uint32_t slot = 0, phase = 0, at = 0;       // the current row's stage, its parity and place
    uint32_t ask_slot = 0;                      // thread 0: the next row's to ask for
    bool dead = false;

    __device__ __forceinline__ void init(unsigned char* shared, int dim, int arrays)
    {
        bars = (uint32_t)__cvta_generic_to_shared(shared);
        data = bars + 64;
        row_bytes = 2 * dim;
        stage_bytes = arrays * row_bytes;
        at = data;
        if (threadIdx.x == 0) {
            for (int i = 0; i < STAGES; ++i) mbar_init(bars + 8 * i, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        // a tensor that is not there reads as zeros
        for (uint32_t i = threadIdx.x * 16; i < STAGES * stage_bytes; i += blockDim.x * 16)
            *reinterpret_cast<uint4*>(shared + 64 + i) = make_uint4(0u, 0u, 0u, 0u);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();
    }
    // thread 0: the next row's copies; `rows` holds the arrays' addresses of that row
    template <int N>
    __device__ __forceinline__ void issue(const uint16_t* const (&rows)[N])
    {
        const uint32_t bar = bars + 8 * ask_slot, to = data + ask_slot * stage_bytes;
        uint32_t bytes = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) bytes += rows[i] ? row_bytes : 0u;
        mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (rows[i])
                asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                                 to + i * row_bytes),
                             "l"(rows[i]), "r"(row_bytes), "r"(bar)
                             : "memory");
        ask_slot = ask_slot + 1 == STAGES ? 0 : ask_slot + 1;
    }
    __device__ __forceinline__ void wait()
    {
        if (!dead && !mbar_wait(bars + 8 * slot, phase, kRowWaitNs)) {
            atomicOr(&g_norm_error, 1u);
            dead = true;
        }
    }
    __device__ __forceinline__ void next()
    {
        if (++slot == STAGES) {
            slot = 0;
            phase ^= 1u;
            at = data;
        } else {
            at += stage_bytes;
        }
    }
    // thread 0, after the last row: a wait that ran out has left copies behind, none may outlive the block
    __device__ __forceinline__ void drain()
    {
        if (!dead) return;
        for (uint32_t i = 0; i < STAGES; ++i) {
            mbar_wait(bars + 8 * i, 0, kRowWaitNs);
            mbar_wait(bars + 8 * i, 1, kRowWaitNs);
        }
    }
    template <int V>
    __device__ __forceinline__ Raw<V> get(int array, const Lane<kEven, V>& L) const
    {
        Raw<V> r;
        const uint32_t from = at + array * row_bytes + L.tid * 16;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            uint4 q;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                         : "r"(from + v * L.T * 16)
                         : "memory");
            r.w[4 * v] = q.x; r.w[4 * v + 1] = q.y; r.w[4 * v + 2] = q.z; r.w[4 * v + 3] = q.w;
        }
        return r;
    }
};

constexpr int pipe_bytes(int64_t dim, int arrays, int stages) { return 64 + stages * arrays * 2 * (int)dim; }

// Forward: threads (T, rows a block); a block of more than one row has T = 32.
template <int DT, int MODE, bool LAYER, int V, bool STAGED>
__global__ void __launch_bounds__(V == 4 ? 256 : 512) block_norm_kernel(const __grid_constant__ NormParams P)
{
    after_earlier_work();
    __shared__ __align__(16) float area[2 * kSumArea];
    extern __shared__ __align__(128) unsigned char stages[];
    const int T = blockDim.x;
    const Lane<MODE, V> L(threadIdx.x, T, P.dim);
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= P.rows) return;                    // whole blocks, or warps that sum by themselves
    int turn = 0;
    RowPipe<kForwardStages> pipe;
    const bool own_gates = P.gate && P.gate_rows == 1;
    auto ask = [&](int64_t r) {
        const uint16_t* const rows[3] = {P.h + r * P.ld_h, P.x ? P.x + r * P.ld_x : nullptr, own_gates ? P.gate + r * P.ld_gate : nullptr};
        pipe.issue(rows);
    };
    if constexpr (STAGED) {
        pipe.init(stages, P.dim, own_gates ? 3 : 2);
        if (threadIdx.x == 0)
            for (int k = 0; k < kForwardStages && row + k * step < P.rows; ++k) ask(row + k * step);
    }
    GateRow at(P.gate ? row : 0, step, P.gate ? P.gate_rows : 1);
    bool first = true;
    for (; row < P.rows; row += step) {
        F2 a[4 * V];
        Raw<V> h, x;
        if constexpr (STAGED) {
            pipe.wait();
            h = pipe.get<V>(0, L);
        } else {
            h = load_raw<MODE, V>(P.h + row * P.ld_h, L);
            if (P.x) x = load_raw<MODE, V>(P.x + row * P.ld_x, L);
        }
#pragma unroll
        for (int k = 0; k < 4 * V; ++k) a[k] = widen<DT>(h.w[k]);
        // every thread is past the first sum: the row before is done with, its stage is free
        auto refill = [&]() {
            if constexpr (STAGED) {
                const int64_t r = row + (kForwardStages - 1) * step;
                if (threadIdx.x == 0 && !first && r < P.rows) ask(r);
                first = false;
            }
        };
        if (P.post) {
            // the weights are fetched before the sums that they wait for
            const Raw<V> w = load_weight<MODE, V>(P.post_w, L), c = load_weight<MODE, V>(P.post_b, L);
            const F2 r = both(centre<LAYER, MODE, V>(a, L, P, T, area, turn));
            refill();
#pragma unroll
            for (int k = 0; k < 4 * V; ++k) a[k] = fma(mul(a[k], r), widen<DT>(w.w[k]), widen<DT>(c.w[k]));
        }
        const F2 scale = both(P.scale);
        if (P.gate) {
            Raw<V> gate;
            if constexpr (STAGED) gate = own_gates ? pipe.get<V>(2, L) : load_raw<MODE, V>(P.gate + at.group * P.ld_gate, L);
            else gate = load_raw<MODE, V>(P.gate + at.group * P.ld_gate, L);
#pragma unroll
            for (int k = 0; k < 4 * V; ++k) a[k] = mul(a[k], mul(scale, widen<DT>(gate.w[k])));
            at.next();
        } else {
#pragma unroll
            for (int k = 0; k < 4 * V; ++k) a[k] = mul(a[k], scale);
        }
        if constexpr (STAGED) x = pipe.get<V>(1, L);
        if (STAGED || P.x) {
#pragma unroll
            for (int k = 0; k < 4 * V; ++k) a[k] = add(a[k], widen<DT>(x.w[k]));
        }
        if (P.y) store_row<DT, MODE, V>(P.y + row * P.ld_y, L, a);
        if (P.pre) {
            if constexpr (MODE != kEven) clear_rest<MODE, V>(L, a);
            const Raw<V> w = load_weight<MODE, V>(P.pre_w, L), c = load_weight<MODE, V>(P.pre_b, L);
            const F2 r = both(centre<LAYER, MODE, V>(a, L, P, T, area, turn));
            if (!P.post) refill();
#pragma unroll
            for (int k = 0; k < 4 * V; ++k) a[k] = fma(mul(a[k], r), widen<DT>(w.w[k]), widen<DT>(c.w[k]));
            store_row<DT, MODE, V>(P.z + row * P.ld_z, L, a);
        }
        if constexpr (STAGED) pipe.next();
    }
    if constexpr (STAGED)
        if (threadIdx.x == 0) pipe.drain();
}

// A worker's sums over its rows, by column: registers, or shared memory.
enum { kPreW = 0, kPostW = 1, kGate = 2, kPreB = 3, kPostB = 4 };
template <bool SHARED, int NACC, int V>
struct Acc {
    F2 v[SHARED ? 1 : NACC][4 * V];
    F2* s;
    int tid, T;
    __device__ __forceinline__ Acc(F2* shared, int tid_, int T_) : s(shared), tid(tid_), T(T_) {}
    __device__ __forceinline__ F2& at(int k, int j)
    {
        if constexpr (SHARED) return s[(k * 4 * V + j) * T + tid];
        else return v[k][j];
    }
    __device__ __forceinline__ void clear(int k)
    {
#pragma unroll
        for (int j = 0; j < 4 * V; ++j) at(k, j) = both(0.0f);
    }
};

// The sums of the biases' gradients are kept where they may be asked for: with ZERO_NORM_LAYER, and
// in the variant with shared memory.
template <int DT, int MODE, bool LAYER, int V, bool SHARED, bool STAGED>
__global__ void __launch_bounds__(V == 2 && !SHARED ? 256 : 512, V == 2 && !SHARED ? 2 : 1)
    block_norm_grad_kernel(const __grid_constant__ NormParams P)
{
    after_earlier_work();
    __shared__ __align__(16) float area[2 * kSumArea];
    extern __shared__ __align__(128) unsigned char stages[];
    constexpr bool BIAS = LAYER || SHARED;
    constexpr int NACC = BIAS ? 5 : 3;
    const int T = blockDim.x;
    const Lane<MODE, V> L(threadIdx.x, T, P.dim);
    const int64_t worker = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int64_t r0 = worker * P.chunk, r1 = min(P.rows, r0 + P.chunk);
    if (r0 >= r1) return;                         // whole blocks, or warps that sum by themselves
    Acc<SHARED, NACC, V> acc(reinterpret_cast<F2*>(stages), threadIdx.x, T);
#pragma unroll
    for (int k = 0; k < 3; ++k) acc.clear(k);
    if constexpr (BIAS)
        if (!SHARED || P.bias_sums)
#pragma unroll
            for (int k = 3; k < 5; ++k) acc.clear(k);
    int turn = 0;
    RowPipe<kBackwardStages> pipe;
    const bool own_gates = P.gate && P.gate_rows == 1;
    auto ask = [&](int64_t r) {
        const uint16_t* const rows[5] = {P.pre ? P.y_in + r * P.ld_y : nullptr, P.pre ? P.dz + r * P.ld_dz : nullptr,
                                         P.h ? P.h + r * P.ld_h : nullptr, P.dy ? P.dy + r * P.ld_dy : nullptr,
                                         own_gates ? P.gate + r * P.ld_gate : nullptr};
        pipe.issue(rows);
    };
    if constexpr (STAGED) {
        pipe.init(stages, P.dim, own_gates ? 5 : 4);
        if (threadIdx.x == 0)
            for (int k = 0; k < kBackwardStages && r0 + k < r1; ++k) ask(r0 + k);
    }
    GateRow at(P.gate_rows ? r0 : 0, 1, P.gate_rows ? P.gate_rows : 1);
    int64_t group_first = r0;                     // the group's first row in the worker
    const F2 scale = both(P.scale);
    auto next_row = [&]() {
        if constexpr (STAGED) pipe.next();
    };
    for (int64_t row = r0; row < r1; ++row, next_row()) {
        Raw<V> hr = {}, yr = {}, zr = {}, dr = {};
        if constexpr (STAGED) {
            pipe.wait();
        } else {
            if (P.pre) {
                yr = load_raw<MODE, V>(P.y_in + row * P.ld_y, L);
                zr = load_raw<MODE, V>(P.dz + row * P.ld_dz, L);
            }
            if (P.h) hr = load_raw<MODE, V>(P.h + row * P.ld_h, L);
            if (P.dy) dr = load_raw<MODE, V>(P.dy + row * P.ld_dy, L);
        }
        auto fetch = [&](int which, const Raw<V>& kept) {
            if constexpr (STAGED) return pipe.get<V>(which, L);
            else return kept;
        };
        // minus the means of y and h
        F2 ma = both(0.0f), mb = both(0.0f);
        auto refill = [&]() {
            // every thread is past the first sum: the row before is done with, its stage is free
            if constexpr (STAGED)
                if (threadIdx.x == 0 && row > r0 && row + kBackwardStages - 1 < r1) ask(row + kBackwardStages - 1);
        };
        if constexpr (LAYER) {
            const Raw<V> h = fetch(2, hr), y = fetch(0, yr);
            F2 sa = both(0.0f), sb = sa;
#pragma unroll
            for (int k = 0; k < 4 * V; ++k) {
                sa = add(sa, widen<DT>(h.w[k]));
                sb = add(sb, widen<DT>(y.w[k]));
            }
            float s[2] = {total(sa), total(sb)};
            row_sum(s, T, area, turn);
            refill();
            ma = both(P.post ? -s[0] * P.inv_dim : 0.0f);
            mb = both(-s[1] * P.inv_dim);
        }
        auto centred = [&](uint32_t w, F2 minus_mean, int k) {
            const F2 x = widen<DT>(w);
            if constexpr (LAYER) {
                const F2 c = add(x, minus_mean);
                return MODE != kEven ? held<MODE, V>(L, k, c) : c;
            } else {
                return x;
            }
        };
        F2 d[4 * V];
        float rh = 1.0f;
        {
            float s[4];
            {
                const Raw<V> h = fetch(2, hr), y = fetch(0, yr), z = fetch(1, zr);
                const Raw<V> w = load_weight<MODE, V>(P.pre_w, L);
                F2 s0 = both(0.0f), s1 = s0, s2 = s0, s3 = s0;
#pragma unroll
                for (int k = 0; k < 4 * V; ++k) {
                    const F2 a = centred(h.w[k], ma, k), b = centred(y.w[k], mb, k), g = mul(widen<DT>(z.w[k]), widen<DT>(w.w[k]));
                    s0 = fma(a, a, s0);
                    s1 = fma(b, b, s1);
                    s2 = fma(g, b, s2);
                    if (LAYER) s3 = add(s3, g);
                }
                s[0] = total(s0);
                s[1] = total(s1);
                s[2] = total(s2);
                s[3] = total(s3);
            }
            if constexpr (LAYER) {
                row_sum(s, T, area, turn);
            } else {
                float t[3] = {s[0], s[1], s[2]};
                row_sum(t, T, area, turn);
                refill();
                s[0] = t[0];
                s[1] = t[1];
                s[2] = t[2];
            }
            if (P.post) rh = rsqrtf(s[0] * P.inv_dim + P.eps);
            const Raw<V> e = fetch(3, dr);
#pragma unroll
            for (int k = 0; k < 4 * V; ++k) d[k] = widen<DT>(e.w[k]);
            if (P.pre) {
                const float ry = rsqrtf(s[1] * P.inv_dim + P.eps);
                const F2 r = both(ry), along = both(-s[2] * P.inv_dim * ry * ry), mean = both(LAYER ? -s[3] * P.inv_dim : 0.0f);
                const Raw<V> y = fetch(0, yr), z = fetch(1, zr), w = load_weight<MODE, V>(P.pre_w, L);
#pragma unroll
                for (int k = 0; k < 4 * V; ++k) {
                    const F2 b = centred(y.w[k], mb, k), c = widen<DT>(z.w[k]);
                    acc.at(kPreW, k) = fma(c, mul(b, r), acc.at(kPreW, k));
                    if constexpr (BIAS)
                        if (!SHARED || P.bias_sums) acc.at(kPreB, k) = add(acc.at(kPreB, k), c);
                    F2 g = fma(c, widen<DT>(w.w[k]), mul(b, along));
                    if (LAYER) g = add(g, mean);
                    d[k] = fma(r, g, d[k]);
                }
            }
        }
        if (P.dx) store_row<DT, MODE, V>(P.dx + row * P.ld_dx, L, d);
        const int64_t group = at.group;
        const bool group_ends = row + 1 == r1 || (P.gate_rows && at.rest + 1 == P.gate_rows);
        at.next();
        if (!P.dh && !P.sums && !P.dgate) continue;
        // through the gate: a is the normalised h (formed anew where it is used, registers are few), d
        // becomes du
        const F2 r_h = both(rh);
        auto normal_h = [&](const Raw<V>& h, int k) { return mul(centred(h.w[k], ma, k), r_h); };
        if (P.dgate) {
            const Raw<V> h = fetch(2, hr), w = load_weight<MODE, V>(P.post_w, L), e = load_weight<MODE, V>(P.post_b, L);
            if (P.gate_rows == 1) {
                F2 u[4 * V];
#pragma unroll
                for (int k = 0; k < 4 * V; ++k)
                    u[k] = mul(mul(scale, d[k]), fma(normal_h(h, k), widen<DT>(w.w[k]), widen<DT>(e.w[k])));
                store_row<DT, MODE, V>(P.dgate + row * P.ld_dgate, L, u);
            } else {
#pragma unroll
                for (int k = 0; k < 4 * V; ++k)
                    acc.at(kGate, k) = fma(mul(scale, d[k]), fma(normal_h(h, k), widen<DT>(w.w[k]), widen<DT>(e.w[k])), acc.at(kGate, k));
                if (group_ends) {
                    // whole groups are final; else a part of one, in the worker's first or last slot
                    const int64_t first = group * P.gate_rows, last = min(P.rows, first + P.gate_rows) - 1;
                    F2 u[4 * V];
#pragma unroll
                    for (int k = 0; k < 4 * V; ++k) u[k] = acc.at(kGate, k);
                    if (first >= r0 && last < r1) {
                        store_row<DT, MODE, V>(P.dgate + group * P.ld_dgate, L, u);
                    } else {
                        store_sums<MODE, V>(P.gate_sums + (worker * 2 + (group_first == r0 ? 0 : 1)) * P.dim, L, u);
                    }
                    acc.clear(kGate);
                    group_first = row + 1;
                }
            }
        }
        if (!P.dh && !P.sums) continue;
        if (P.gate) {
            Raw<V> gate;
            if constexpr (STAGED) gate = own_gates ? pipe.get<V>(4, L) : load_raw<MODE, V>(P.gate + group * P.ld_gate, L);
            else gate = load_raw<MODE, V>(P.gate + group * P.ld_gate, L);
#pragma unroll
            for (int k = 0; k < 4 * V; ++k) d[k] = mul(d[k], mul(scale, widen<DT>(gate.w[k])));
        } else {
#pragma unroll
            for (int k = 0; k < 4 * V; ++k) d[k] = mul(d[k], scale);
        }
        if (P.post) {
            F2 s0 = both(0.0f), s1 = s0;
            {
                const Raw<V> h = fetch(2, hr), w = load_weight<MODE, V>(P.post_w, L);
#pragma unroll
                for (int k = 0; k < 4 * V; ++k) {
                    const F2 a = normal_h(h, k);
                    acc.at(kPostW, k) = fma(d[k], a, acc.at(kPostW, k));
                    if constexpr (BIAS)
                        if (!SHARED || P.bias_sums) acc.at(kPostB, k) = add(acc.at(kPostB, k), d[k]);
                    d[k] = mul(d[k], widen<DT>(w.w[k]));
                    if constexpr (MODE != kEven) d[k] = held<MODE, V>(L, k, d[k]);
                    s0 = fma(d[k], a, s0);
                    if (LAYER) s1 = add(s1, d[k]);
                }
            }
            float t[2] = {total(s0), total(s1)};
            if constexpr (LAYER) {
                row_sum(t, T, area, turn);
            } else {
                float one[1] = {t[0]};
                row_sum(one, T, area, turn);
                t[0] = one[0];
            }
            const F2 along = both(-t[0] * P.inv_dim * rh), mean = both(LAYER ? -t[1] * P.inv_dim * rh : 0.0f);
            const Raw<V> h = fetch(2, hr);
#pragma unroll
            for (int k = 0; k < 4 * V; ++k) {
                F2 g = mul(normal_h(h, k), along);
                if (LAYER) g = add(g, mean);
                d[k] = fma(r_h, d[k], g);
            }
        }
        if (P.dh) store_row<DT, MODE, V>(P.dh + row * P.ld_dh, L, d);
    }
    if (P.sums) {
        float* q = P.sums + worker * 4 * P.dim;
        F2 t[4 * V];
        auto put = [&](int k, int row) {
#pragma unroll
            for (int j = 0; j < 4 * V; ++j) t[j] = acc.at(k, j);
            store_sums<MODE, V>(q + row * P.dim, L, t);
        };
        put(kPreW, 0);
        put(kPostW, 2);
        if constexpr (BIAS)
            if (P.bias_sums) {
                put(kPreB, 1);
                put(kPostB, 3);
            }
    }
    if constexpr (STAGED)
        if (threadIdx.x == 0) pipe.drain();
}

struct SumParams {
    const float* sums;
    const float* gate_sums;
    uint16_t* out[4];          // dpre_w, dpre_b, dpost_w, dpost_b, or NULL
    uint16_t* dgate;
    int64_t rows, ld_dgate, gate_rows, chunk, workers;
    int32_t dim;
    int32_t by_group;          // gate sums: one place a group, or a worker
    int32_t apart;             // kSumLanes places a block row, or one
};

constexpr int kSumLanes = 16;

// Block (column chunk, j): j < 4 adds the workers' sums of one weight, kSumLanes workers at a time; then come
// the gate groups that span workers, kSumLanes a block (`apart`, where a group has no more workers than
// that: one thread adds them in order) or one a block.  Four columns a thread where dim allows.  The order
// is fixed.  A worker's sums are read once; what bounds it is the number of loads in flight: 304 workers of
// 4096 columns 8.5 us (8 lanes 16), 501 of 1023 and 143 groups 8.5 (8 lanes, a block a group 13).
template <int DT, int C>
__global__ void __launch_bounds__(32 * kSumLanes) block_norm_sum_kernel(const __grid_constant__ SumParams P)
{
    after_earlier_work();
    __shared__ float part[kSumLanes][32 * C + 1];
    const int col = (blockIdx.x * 32 + threadIdx.x) * C, lane = threadIdx.y;
    const float* from;
    int64_t w0, w1, stride;
    uint16_t* out = nullptr;
    bool later = false;        // the group starts after its first worker's first row: the second slot
    const bool weight = blockIdx.y < 4, apart = !weight && P.apart;
    if (weight) {
        out = P.out[blockIdx.y];
        from = P.sums + (int64_t)blockIdx.y * P.dim;
        stride = 4 * P.dim;
        w0 = 0;
        w1 = P.workers - 1;
    } else {
        const int64_t i = apart ? (int64_t)(blockIdx.y - 4) * kSumLanes + lane : blockIdx.y - 4;
        const int64_t group = P.by_group ? i : (min(P.rows, (i + 1) * P.chunk) - 1) / P.gate_rows;
        const int64_t first = group * P.gate_rows, last = min(P.rows, first + P.gate_rows) - 1;
        w0 = first / P.chunk;
        w1 = last / P.chunk;
        // else it is whole in one worker, or another block's
        if (P.dgate && first < P.rows && w0 != w1 && (P.by_group || w0 == i)) out = P.dgate + group * P.ld_dgate;
        from = P.gate_sums;
        stride = 2 * P.dim;
        later = first > w0 * P.chunk;
    }
    if (!apart && !out) return;
    float s[C];
#pragma unroll
    for (int c = 0; c < C; ++c) s[c] = 0.0f;
    if (col < P.dim && out) {
        const int64_t step = apart ? 1 : kSumLanes;
        auto add = [&](const float* q) {
            if constexpr (C == 4) {
                const float4 f = *reinterpret_cast<const float4*>(q);
                s[0] += f.x; s[1] += f.y; s[2] += f.z; s[3] += f.w;
            } else {
                s[0] += *q;
            }
        };
        int64_t w = apart ? w0 : w0 + lane;
        if (later && w == w0) {
            add(from + w * stride + P.dim + col);
            w += step;
        }
#pragma unroll 8
        for (; w <= w1; w += step) add(from + w * stride + col);
    }
    if (apart) {
        if (col < P.dim && out)
#pragma unroll
            for (int c = 0; c < C; ++c) out[col + c] = narrow1<DT>(s[c]);
        return;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) part[lane][threadIdx.x * C + c] = s[c];
    __syncthreads();
    const int i = lane * 32 + threadIdx.x, e = blockIdx.x * 32 * C + i;
    if (i < 32 * C && e < P.dim) {
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < kSumLanes; ++k) sum += part[k][i];
        out[e] = narrow1<DT>(sum);
    }
}

// ------------------------------------------------------------------ host

constexpr int kSms = 152;
constexpr int kForwardMost = 4;
constexpr int kForwardThreads = 1024;             // an SM's, of the staged forward kernel

// How a row is held: V eights a thread in T threads.  The sums over a row cost the same instructions
// whatever a thread holds, so more elements a thread are better while registers last: 32 forward (16
// where they come one by one), 16 backward (whose column sums take two and a half times as many
// registers again).
struct Hold {
    int V = 1, T = 32;
    bool even = true;          // every thread holds as much
};

Hold hold_row(int64_t dim, int most)
{
    Hold best;
    for (int V = most; V >= 1; V /= 2) {
        Hold h;
        h.V = V;
        h.T = (int)((dim + 8 * V * 32 - 1) / (8 * V * 32)) * 32;
        h.even = (int64_t)h.T * 8 * V == dim;
        // fewer idle places, in blocks that their kernels are built for
        if (V == most || (h.T <= 256 && (int64_t)h.T * h.V < (int64_t)best.T * best.V)) best = h;
    }
    return best;
}

// How the backward pass cuts the rows: workers of `chunk` consecutive ones.
struct Cut {
    Hold hold;
    int per_block = 1;
    bool shared = false;
    int64_t chunk = 1, workers = 0;
};

Cut cut_rows(const zero_block_norm_t& a)
{
    Cut c;
    const bool layer = a.kind == ZERO_NORM_LAYER;
    // five column sums leave registers for eight elements a thread, three for sixteen
    c.hold = hold_row(a.dim, a.dim <= 256 || (layer && a.dim <= 4096) ? 1 : 2);
    // more than 4096 elements (their threads' registers do not hold the column sums), and the biases'
    // gradients of an RMS norm (the register variant keeps none)
    c.shared = a.dim > 4096 || (!layer && (a.dpre_b || a.dpost_b));
    if (c.shared) c.hold = hold_row(a.dim, 2);
    c.per_block = c.hold.T == 32 && !c.shared ? 8 : 1;
    const int blocks_per_sm = std::max(1, 512 / (c.hold.T * c.per_block));
    const int64_t most = (int64_t)kSms * blocks_per_sm * c.per_block;
    c.chunk = std::max<int64_t>(1, (a.rows + most - 1) / most);
    // chunks that end with gate groups where that costs little balance
    const int64_t R = a.rows_per_gate;
    if (R > 1 && c.chunk % R != 0) {
        const int64_t rounded = (c.chunk + R - 1) / R * R;
        if (rounded * 8 <= c.chunk * 9) c.chunk = rounded;
    }
    c.workers = (a.rows + c.chunk - 1) / c.chunk;
    return c;
}

struct Checked {
    zero_block_norm_t a;
    bool vec = true;
    Cut cut;
    int64_t groups = 0, sums_bytes = 0, gate_bytes = 0;
};

zero_status_t check_norm(const zero_block_norm_t* in, bool back, Checked* C, const char* who)
{
    const std::string w = std::string(who) + ": ";
    if (!in) return fail(ZERO_EINVAL, w + "NULL arguments");
    C->a = *in;
    zero_block_norm_t& a = C->a;
    if (a.rows < 0 || a.dim < 1) return fail(ZERO_EINVAL, w + "bad size");
    if (a.dim > ZERO_NORM_MAX_DIM) return fail(ZERO_ERANGE, w + "dim beyond ZERO_NORM_MAX_DIM");
    if (a.rows > ((int64_t)1 << 40)) return fail(ZERO_ERANGE, w + "rows beyond 2^40");
    if (a.dtype16 != ZERO_BF16 && a.dtype16 != ZERO_FP16) return fail(ZERO_EINVAL, w + "bad dtype16");
    if (a.kind != ZERO_NORM_RMS && a.kind != ZERO_NORM_LAYER) return fail(ZERO_EINVAL, w + "bad kind");
    if (a.norms & ~(ZERO_NORM_PRE | ZERO_NORM_POST)) return fail(ZERO_EINVAL, w + "bad norms");
    if (!(a.eps >= 0.0) || !std::isfinite(a.eps) || !std::isfinite(a.residual_scale))
        return fail(ZERO_EINVAL, w + "bad eps or residual_scale");
    if (a.rows_per_gate < 0 || (a.rows > 0 && (a.rows_per_gate == 0) != (a.gate == nullptr)))
        return fail(ZERO_EINVAL, w + "a gate needs rows_per_gate >= 1, and none 0");
    // more rows than there are: one gate row for all (rows that share one are added up below)
    if (a.rows_per_gate > a.rows) a.rows_per_gate = std::max<int64_t>(1, a.rows);
    const bool pre = a.norms & ZERO_NORM_PRE, post = a.norms & ZERO_NORM_POST;
    C->groups = a.rows_per_gate ? (a.rows + a.rows_per_gate - 1) / a.rows_per_gate : 0;
    int64_t* lds[] = {&a.ld_h, &a.ld_x, &a.ld_y, &a.ld_z, &a.ld_gate, &a.ld_dy, &a.ld_dz, &a.ld_dx, &a.ld_dh, &a.ld_dgate};
    for (int64_t* ld : lds) {
        if (*ld == 0) *ld = a.dim;
        if (*ld < a.dim) return fail(ZERO_EINVAL, w + "a row stride is shorter than its row");
        if (*ld > ((int64_t)1 << 38)) return fail(ZERO_ERANGE, w + "a row stride beyond 2^38");
    }
    const void* every[] = {a.h, a.x, a.gate, a.post_w, a.post_b, a.pre_w, a.pre_b, a.y, a.z, a.dy, a.dz, a.dx, a.dh, a.dgate,
                           a.dpost_w, a.dpost_b, a.dpre_w, a.dpre_b};
    for (const void* p : every)
        if (!aligned(p, 2)) return fail(ZERO_EALIGN, w + "a pointer is not aligned to 2 bytes");
    if (!back) {
        if (a.rows > 0 && !a.h) return fail(ZERO_EINVAL, w + "h is NULL");
        if (a.rows > 0 && pre && !a.z) return fail(ZERO_EINVAL, w + "z is NULL");
        if (a.rows > 0 && !pre && !a.y) return fail(ZERO_EINVAL, w + "no output");
        if (a.y && ((a.y == a.x && a.ld_y != a.ld_x) || a.y == a.h || (pre && a.y == a.z)))
            return fail(ZERO_EINVAL, w + "y overlaps another buffer");
        if (pre && a.z && ((a.z == a.h && a.ld_z != a.ld_h) || a.z == a.x)) return fail(ZERO_EINVAL, w + "z overlaps another buffer");
    } else {
        if (a.rows > 0 && pre && (!a.y || !a.dz)) return fail(ZERO_EINVAL, w + "the pre-norm's gradient needs y and dz");
        if (a.rows > 0 && !a.h && ((post && (a.dh || a.dpost_w)) || a.dgate))
            return fail(ZERO_EINVAL, w + "h is NULL");
        if (!pre && (a.dpre_w || a.dpre_b)) return fail(ZERO_EINVAL, w + "gradients of a pre-norm that is not there");
        if (!post && (a.dpost_w || a.dpost_b)) return fail(ZERO_EINVAL, w + "gradients of a post-norm that is not there");
        if (a.rows > 0 && a.dgate && !a.gate) return fail(ZERO_EINVAL, w + "the gradient of a gate that is not there");
        if (!a.dx && !a.dh && !a.dgate && !a.dpost_w && !a.dpost_b && !a.dpre_w && !a.dpre_b)
            return fail(ZERO_EINVAL, w + "no gradient asked for");
        if (a.dx && ((a.dx == a.dy && a.ld_dx != a.ld_dy) || a.dx == a.dz || a.dx == a.h || a.dx == a.y || a.dx == a.dh))
            return fail(ZERO_EINVAL, w + "dx overlaps another buffer");
        C->cut = cut_rows(a);
        const bool weights = a.dpre_w || a.dpre_b || a.dpost_w || a.dpost_b;
        if (weights) C->sums_bytes = C->cut.workers * 4 * a.dim * 4;
        if (a.dgate && a.rows_per_gate > 1) C->gate_bytes = C->cut.workers * 2 * a.dim * 4;
    }
    // 16-byte accesses need every row of every tensor in use to start on 16 bytes
    C->vec = a.dim % 8 == 0;
    struct {
        const void* p;
        int64_t ld;
    } rowsets[] = {{a.h, a.ld_h}, {back ? nullptr : a.x, a.ld_x}, {a.gate, a.ld_gate}, {a.y, a.ld_y}, {back ? nullptr : a.z, a.ld_z},
                   {back ? a.dy : nullptr, a.ld_dy}, {back ? a.dz : nullptr, a.ld_dz}, {back ? a.dx : nullptr, a.ld_dx},
                   {back ? a.dh : nullptr, a.ld_dh}, {back ? a.dgate : nullptr, a.ld_dgate},
                   {a.post_w, 0}, {a.post_b, 0}, {a.pre_w, 0}, {a.pre_b, 0}};
    for (const auto& r : rowsets)
        if (r.p && (!aligned(r.p, 16) || r.ld % 8 != 0)) C->vec = false;
    return ZERO_OK;
}

// The address of g_no_weights on the current device.
const uint16_t* no_weights()
{
    static std::mutex mu;
    static const void* cache[64] = {nullptr};
    int dev = 0;
    void* p = nullptr;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (!cache[dev] && cudaGetSymbolAddress(&p, g_no_weights) == cudaSuccess) cache[dev] = p;
    return static_cast<const uint16_t*>(cache[dev]);
}

NormParams params_of(const Checked& C, bool back)
{
    const zero_block_norm_t& a = C.a;
    NormParams P;
    std::memset(&P, 0, sizeof(P));
    auto in = [](const void* p) { return static_cast<const uint16_t*>(p); };
    auto out = [](void* p) { return static_cast<uint16_t*>(p); };
    P.post = (a.norms & ZERO_NORM_POST) != 0;
    P.pre = (a.norms & ZERO_NORM_PRE) != 0;
    P.h = in(a.h);
    P.gate = in(a.gate);
    const uint16_t* none = no_weights();
    auto weights = [&](const void* p, int which) { return p ? Weights{in(p), 0xFFFFFFFFu} : Weights{none + 8 * which, 0u}; };
    const int ones = a.dtype16 == ZERO_BF16 ? 0 : 1;
    P.post_w = weights(P.post ? a.post_w : nullptr, ones);
    P.post_b = weights(P.post ? a.post_b : nullptr, 2);
    P.pre_w = weights(P.pre ? a.pre_w : nullptr, ones);
    P.pre_b = weights(P.pre ? a.pre_b : nullptr, 2);
    if (back) {
        P.y_in = in(a.y);
        P.dy = in(a.dy);
        P.dz = P.pre ? in(a.dz) : nullptr;
        P.dx = out(a.dx);
        P.dh = out(a.dh);
        P.dgate = out(a.dgate);
        // h only where the post-norm or the gate's gradient uses it
        if (!P.post && !P.dgate) P.h = nullptr;
    } else {
        P.x = in(a.x);
        P.y = out(a.y);
        P.z = out(a.z);
    }
    P.rows = a.rows;
    P.ld_h = a.ld_h;
    P.ld_x = a.ld_x;
    P.ld_y = a.ld_y;
    P.ld_z = a.ld_z;
    P.ld_gate = a.ld_gate;
    P.ld_dy = a.ld_dy;
    P.ld_dz = a.ld_dz;
    P.ld_dx = a.ld_dx;
    P.ld_dh = a.ld_dh;
    P.ld_dgate = a.ld_dgate;
    P.gate_rows = a.rows_per_gate;
    P.dim = (int32_t)a.dim;
    P.eps = (float)a.eps;
    P.scale = (float)a.residual_scale;
    P.inv_dim = (float)(1.0 / (double)a.dim);
    return P;
}

constexpr int kMostShared = 227 * 1024 - 1024;   // beside the kernels' static shared memory

template <auto KERNEL>
zero_status_t launch(unsigned grid, dim3 threads, int64_t bytes, const NormParams& P, cudaStream_t s)
{
    if (bytes > 48 * 1024) {
        const cudaError_t set = allow_shared<KERNEL>(kMostShared);
        if (set != cudaSuccess) return cuda_fail(set, "zero_block_norm: shared memory");
    }
    launch_after(KERNEL, grid, threads, (size_t)bytes, s, P);
    return ZERO_OK;
}

template <int DT, int MODE, bool LAYER>
zero_status_t launch_forward(const NormParams& P, const Hold& h, cudaStream_t s)
{
    const int per_block = h.T == 32 ? 8 : 1;
    const int64_t blocks = (P.rows + per_block - 1) / per_block;
    const dim3 threads(h.T, per_block);
    if constexpr (MODE == kEven) {
        // a row of its own a block, and more rows than the GPU takes at once: through shared memory
        const int64_t bytes = pipe_bytes(P.dim, P.gate && P.gate_rows == 1 ? 3 : 2, kForwardStages);
        if (h.T > 32 && (P.pre || P.post) && P.rows > 4 * kSms) {
            const int64_t fit = std::min<int64_t>(kMostShared / (bytes + 2048), kForwardThreads / h.T);
            const unsigned grid = (unsigned)std::min<int64_t>(blocks, kSms * std::max<int64_t>(1, fit));
            if (h.V == 4) return launch<block_norm_kernel<DT, MODE, LAYER, 4, true>>(grid, threads, bytes, P, s);
            if (h.V == 2) return launch<block_norm_kernel<DT, MODE, LAYER, 2, true>>(grid, threads, bytes, P, s);
            return launch<block_norm_kernel<DT, MODE, LAYER, 1, true>>(grid, threads, bytes, P, s);
        }
    }
    const unsigned grid = (unsigned)std::min<int64_t>(blocks, (int64_t)kSms * std::max(1, 1024 / (h.T * per_block)));
    if constexpr (MODE != kScalar)
        if (h.V == 4) return launch<block_norm_kernel<DT, MODE, LAYER, 4, false>>(grid, threads, 0, P, s);
    if (h.V == 2) return launch<block_norm_kernel<DT, MODE, LAYER, 2, false>>(grid, threads, 0, P, s);
    return launch<block_norm_kernel<DT, MODE, LAYER, 1, false>>(grid, threads, 0, P, s);
}

template <int DT, int MODE, bool LAYER>
zero_status_t launch_backward(const NormParams& P, const Cut& c, cudaStream_t s)
{
    const dim3 threads(c.hold.T, c.per_block);
    const unsigned grid = (unsigned)((c.workers + c.per_block - 1) / c.per_block);
    if (c.shared) {
        const int64_t bytes = (int64_t)(P.bias_sums ? 5 : 3) * 8 * c.hold.V * c.hold.T * 4;
        if (c.hold.V == 2) return launch<block_norm_grad_kernel<DT, MODE, LAYER, 2, true, false>>(grid, threads, bytes, P, s);
        return launch<block_norm_grad_kernel<DT, MODE, LAYER, 1, true, false>>(grid, threads, bytes, P, s);
    }
    if constexpr (MODE == kEven) {
        if (c.hold.T > 32 && (P.pre || P.post) && P.chunk > 1) {
            const int64_t bytes = pipe_bytes(P.dim, P.gate && P.gate_rows == 1 ? 5 : 4, kBackwardStages);
            if constexpr (!LAYER)
                if (c.hold.V == 2) return launch<block_norm_grad_kernel<DT, MODE, LAYER, 2, false, true>>(grid, threads, bytes, P, s);
            return launch<block_norm_grad_kernel<DT, MODE, LAYER, 1, false, true>>(grid, threads, bytes, P, s);
        }
    }
    if constexpr (!LAYER)
        if (c.hold.V == 2) return launch<block_norm_grad_kernel<DT, MODE, LAYER, 2, false, false>>(grid, threads, 0, P, s);
    return launch<block_norm_grad_kernel<DT, MODE, LAYER, 1, false, false>>(grid, threads, 0, P, s);
}

template <int DT, int MODE>
zero_status_t launch_norm(const NormParams& P, const Checked& C, bool back, const Hold& h, cudaStream_t s)
{
    if (C.a.kind == ZERO_NORM_LAYER)
        return back ? launch_backward<DT, MODE, true>(P, C.cut, s) : launch_forward<DT, MODE, true>(P, h, s);
    return back ? launch_backward<DT, MODE, false>(P, C.cut, s) : launch_forward<DT, MODE, false>(P, h, s);
}

template <int DT>
zero_status_t launch_norm(const NormParams& P, const Checked& C, bool back, cudaStream_t s)
{
    const Hold h = back ? C.cut.hold : hold_row(P.dim, C.vec ? kForwardMost : 2);
    if (!C.vec) return launch_norm<DT, kScalar>(P, C, back, h, s);
    return h.even ? launch_norm<DT, kEven>(P, C, back, h, s) : launch_norm<DT, kRagged>(P, C, back, h, s);
}

}  // namespace

cudaError_t take_norm_error(uint32_t* word, void* stream) { return take_error_word(g_norm_error, word, static_cast<cudaStream_t>(stream)); }

}  // namespace zero

using namespace zero;

extern "C" {

zero_status_t zero_block_norm(const zero_block_norm_t* args, void* stream)
try {
    Checked C;
    zero_status_t st = check_norm(args, false, &C, "zero_block_norm");
    if (st != ZERO_OK) return st;
    if (C.a.rows == 0) return ZERO_OK;
    const NormParams P = params_of(C, false);
    if (!P.post_w.p) return fail(ZERO_ECUDA, "zero_block_norm: no device");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    st = C.a.dtype16 == ZERO_BF16 ? launch_norm<ZERO_BF16>(P, C, false, s) : launch_norm<ZERO_FP16>(P, C, false, s);
    if (st != ZERO_OK) return st;
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "zero_block_norm: launch");
}
catch (...) {
    return exception_status("zero_block_norm");
}

zero_status_t zero_block_norm_workspace(const zero_block_norm_t* args, int64_t* bytes)
try {
    if (!bytes) return fail(ZERO_EINVAL, "zero_block_norm_workspace: NULL argument");
    Checked C;
    const zero_status_t st = check_norm(args, true, &C, "zero_block_norm_workspace");
    if (st == ZERO_OK) *bytes = C.sums_bytes + C.gate_bytes;
    return st;
}
catch (...) {
    return exception_status("zero_block_norm_workspace");
}

zero_status_t zero_block_norm_backward(const zero_block_norm_t* args, void* workspace, int64_t workspace_bytes, void* stream)
try {
    Checked C;
    zero_status_t st = check_norm(args, true, &C, "zero_block_norm_backward");
    if (st != ZERO_OK) return st;
    const zero_block_norm_t& a = C.a;
    const int64_t need = C.sums_bytes + C.gate_bytes;
    if (need > 0) {
        if (!workspace) return fail(ZERO_EINVAL, "zero_block_norm_backward: workspace is NULL");
        if (!aligned(workspace, 16)) return fail(ZERO_EALIGN, "zero_block_norm_backward: workspace not 16-byte aligned");
        if (workspace_bytes < need) return fail(ZERO_ERANGE, "zero_block_norm_backward: workspace too small");
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    NormParams P = params_of(C, true);
    P.chunk = C.cut.chunk;
    P.sums = C.sums_bytes ? static_cast<float*>(workspace) : nullptr;
    P.gate_sums = C.gate_bytes ? reinterpret_cast<float*>(static_cast<char*>(workspace) + C.sums_bytes) : nullptr;
    P.bias_sums = a.dpre_b || a.dpost_b;
    const bool bf = a.dtype16 == ZERO_BF16;
    if (a.rows > 0) {
        if (!P.post_w.p) return fail(ZERO_ECUDA, "zero_block_norm_backward: no device");
        st = bf ? launch_norm<ZERO_BF16>(P, C, true, s) : launch_norm<ZERO_FP16>(P, C, true, s);
        if (st != ZERO_OK) return st;
    }
    const bool weights = a.dpre_w || a.dpre_b || a.dpost_w || a.dpost_b, gates = a.rows > 0 && C.gate_bytes > 0;
    if (weights || gates) {
        SumParams S;
        std::memset(&S, 0, sizeof(S));
        S.sums = P.sums;
        S.gate_sums = P.gate_sums;
        S.out[0] = static_cast<uint16_t*>(a.dpre_w);
        S.out[1] = static_cast<uint16_t*>(a.dpre_b);
        S.out[2] = static_cast<uint16_t*>(a.dpost_w);
        S.out[3] = static_cast<uint16_t*>(a.dpost_b);
        S.dgate = gates ? static_cast<uint16_t*>(a.dgate) : nullptr;
        S.rows = a.rows;
        S.ld_dgate = a.ld_dgate;
        S.gate_rows = a.rows_per_gate;
        S.chunk = C.cut.chunk;
        S.workers = C.cut.workers;
        S.dim = (int32_t)a.dim;
        S.by_group = C.groups <= C.cut.workers;
        // a group's workers: at most its rows in chunks, and one more
        S.apart = (a.rows_per_gate + C.cut.chunk - 1) / C.cut.chunk + 1 <= kSumLanes;
        const int64_t places = gates ? std::min(C.groups, C.cut.workers) : 0;
        const unsigned rows = (unsigned)(4 + (S.apart ? (places + kSumLanes - 1) / kSumLanes : places));
        const int cols = a.dim % 4 == 0 ? 128 : 32;
        const dim3 grid((unsigned)((a.dim + cols - 1) / cols), rows), threads(32, kSumLanes);
        if (cols == 128) {
            if (bf) launch_after(block_norm_sum_kernel<ZERO_BF16, 4>, grid, threads, 0, s, S);
            else launch_after(block_norm_sum_kernel<ZERO_FP16, 4>, grid, threads, 0, s, S);
        } else {
            if (bf) launch_after(block_norm_sum_kernel<ZERO_BF16, 1>, grid, threads, 0, s, S);
            else launch_after(block_norm_sum_kernel<ZERO_FP16, 1>, grid, threads, 0, s, S);
        }
    }
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "zero_block_norm_backward: launch");
}
catch (...) {
    return exception_status("zero_block_norm_backward");
}

}  // extern "C"
