// zero_norm.cu -- the norm after one block and the norm before the next, with the block's gate and
// residual scale, and their gradients (zero_block_norm_*):
//   u = Norm_post(h);  y = x + s gate u;  z = Norm_pre(y)
//
// A row is held in registers, eight elements a thread, from its only read to its only write: 8
// bytes an element forward (h, x, y, z), 12 backward (h, y, dy, dz, dx, dh; the statistics are
// formed again from h and y, which are read anyway).  Bound by HBM; the next row is fetched before
// the sums of the current one are formed.  Sums over a row are warp shuffles and one exchange
// through shared memory.
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

struct NormParams {
    const uint16_t *h, *x, *gate, *post_w, *post_b, *pre_w, *pre_b, *dy, *dz;
    const uint16_t* y_in;
    uint16_t *y, *z, *dx, *dh, *dgate;
    int64_t rows, ld_h, ld_x, ld_y, ld_z, ld_gate, ld_dy, ld_dz, ld_dx, ld_dh, ld_dgate;
    int64_t gate_rows;         // rows that share a gate row
    float* sums;               // [worker][4][dim]: dpre_w, dpre_b, dpost_w, dpost_b
    float* gate_sums;          // [worker][2][dim]: a gate group's part in the worker's first / last rows
    int64_t chunk;             // backward: consecutive rows a worker takes
    int32_t dim, post, pre;
    float eps, scale, inv_dim;
};

// Which eight elements of a row a thread holds: neighbours where every row starts on 16 bytes, else
// every T-th, so that a warp's accesses are to neighbouring elements either way.
template <bool VEC>
struct Lane {
    int tid, T, n;             // n: elements held
    __device__ __forceinline__ Lane(int tid_, int T_, int dim) : tid(tid_), T(T_)
    {
        if constexpr (VEC) n = tid * 8 < dim ? 8 : 0;
        else n = tid < dim ? min(8, (dim - tid + T - 1) / T) : 0;
    }
    __device__ __forceinline__ int at(int j) const { return VEC ? tid * 8 + j : tid + j * T; }
};

// Eight 16-bit elements as loaded.
struct Raw {
    uint32_t w[4];
};

template <bool VEC>
__device__ __forceinline__ Raw load_raw(const uint16_t* p, const Lane<VEC>& L)
{
    Raw r;
    if constexpr (VEC) {
        const uint4 q = L.n ? *reinterpret_cast<const uint4*>(p + L.tid * 8) : make_uint4(0u, 0u, 0u, 0u);
        r.w[0] = q.x; r.w[1] = q.y; r.w[2] = q.z; r.w[3] = q.w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t lo = 2 * j < L.n ? p[L.at(2 * j)] : 0u, hi = 2 * j + 1 < L.n ? p[L.at(2 * j + 1)] : 0u;
            r.w[j] = lo | (hi << 16);
        }
    }
    return r;
}

template <int DT>
__device__ __forceinline__ void widen8(const Raw& r, float (&x)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) widen2<DT>(r.w[j], x[2 * j], x[2 * j + 1]);
}

// An optional vector of weights: `other` where there is none.
template <int DT, bool VEC>
__device__ __forceinline__ Raw load_weight(const uint16_t* p, const Lane<VEC>& L, float other)
{
    if (p) return load_raw<VEC>(p, L);
    const uint32_t w = narrow2<DT>(other, other);
    return Raw{{w, w, w, w}};
}

template <int DT, bool VEC>
__device__ __forceinline__ void store_row(uint16_t* p, const Lane<VEC>& L, const float (&x)[8])
{
    if constexpr (VEC) {
        if (L.n)
            *reinterpret_cast<uint4*>(p + L.tid * 8) = make_uint4(narrow2<DT>(x[0], x[1]), narrow2<DT>(x[2], x[3]),
                                                                  narrow2<DT>(x[4], x[5]), narrow2<DT>(x[6], x[7]));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < L.n) p[L.at(j)] = narrow1<DT>(x[j]);
    }
}

// Sums of NV values over the T threads of a row, the same bits in every thread.  `turn` picks one
// of two areas, so that one barrier a sum is enough.
constexpr int kSumArea = 4 * 32;
template <int NV>
__device__ __forceinline__ void row_sum(float (&v)[NV], int T, float* area, int& turn)
{
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
    if (T <= 32) return;
    float* s = area + turn * kSumArea;
    turn ^= 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = T >> 5;
    if (lane == 0)
#pragma unroll
        for (int k = 0; k < NV; ++k) s[k * 32 + warp] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        v[k] = lane < warps ? s[k * 32 + lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
    }
}

// x centred (LAYER) in place, and 1 / sqrt(mean square + eps).
template <bool LAYER, bool VEC>
__device__ __forceinline__ float centre(float (&x)[8], const Lane<VEC>& L, const NormParams& P, int T, float* area, int& turn)
{
    float s[1];
    if constexpr (LAYER) {
        s[0] = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) s[0] += x[j];
        row_sum(s, T, area, turn);
        const float mean = s[0] * P.inv_dim;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = j < L.n ? x[j] - mean : 0.0f;
    }
    s[0] = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s[0] = fmaf(x[j], x[j], s[0]);
    row_sum(s, T, area, turn);
    return rsqrtf(s[0] * P.inv_dim + P.eps);
}

// Forward: threads (T, rows a block); a block of more than one row has T = 32.
template <int DT, bool VEC, bool LAYER, int MOST>
__global__ void __launch_bounds__(MOST) block_norm_kernel(const __grid_constant__ NormParams P)
{
    __shared__ float area[2 * kSumArea];
    const int T = blockDim.x;
    const Lane<VEC> L(threadIdx.x, T, P.dim);
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= P.rows) return;                    // whole blocks, or warps that sum by themselves
    const Raw post_w = load_weight<DT, VEC>(P.post_w, L, 1.0f), post_b = load_weight<DT, VEC>(P.post_b, L, 0.0f);
    const Raw pre_w = load_weight<DT, VEC>(P.pre_w, L, 1.0f), pre_b = load_weight<DT, VEC>(P.pre_b, L, 0.0f);
    int turn = 0;
    Raw h = load_raw<VEC>(P.h + row * P.ld_h, L), x = {}, gate = {};
    if (P.x) x = load_raw<VEC>(P.x + row * P.ld_x, L);
    int64_t group = 0;
    if (P.gate) {
        group = row / P.gate_rows;
        gate = load_raw<VEC>(P.gate + group * P.ld_gate, L);
    }
    for (; row < P.rows; row += step) {
        float a[8], b[8], w[8];
        widen8<DT>(h, a);
        widen8<DT>(x, b);
        float g[8];
        if (P.gate) widen8<DT>(gate, g);
        if (row + step < P.rows) {
            h = load_raw<VEC>(P.h + (row + step) * P.ld_h, L);
            if (P.x) x = load_raw<VEC>(P.x + (row + step) * P.ld_x, L);
            if (P.gate) {
                const int64_t next = (row + step) / P.gate_rows;
                if (next != group) gate = load_raw<VEC>(P.gate + next * P.ld_gate, L);
                group = next;
            }
        }
        if (P.post) {
            const float r = centre<LAYER, VEC>(a, L, P, T, area, turn);
            widen8<DT>(post_w, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] = a[j] * r * w[j];
            widen8<DT>(post_b, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] += w[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = fmaf(P.gate ? P.scale * g[j] : P.scale, a[j], b[j]);
        if (P.y) store_row<DT, VEC>(P.y + row * P.ld_y, L, a);
        if (P.pre) {
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] = j < L.n ? a[j] : 0.0f;
            const float r = centre<LAYER, VEC>(a, L, P, T, area, turn);
            widen8<DT>(pre_w, w);
            widen8<DT>(pre_b, b);
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] = fmaf(a[j] * r, w[j], b[j]);
            store_row<DT, VEC>(P.z + row * P.ld_z, L, a);
        }
    }
}

// A worker's sums over its rows, eight columns a thread: registers, or shared memory.
enum { kPreW = 0, kPostW = 1, kGate = 2, kPreB = 3, kPostB = 4 };
template <bool SHARED, int NACC>
struct Acc {
    float v[SHARED ? 1 : NACC][8];
    float* s;
    int tid, T;
    __device__ __forceinline__ Acc(float* shared, int tid_, int T_) : s(shared), tid(tid_), T(T_)
    {
#pragma unroll
        for (int k = 0; k < NACC; ++k) clear(k);
    }
    __device__ __forceinline__ float& at(int k, int j)
    {
        if constexpr (SHARED) return s[(k * 8 + j) * T + tid];
        else return v[k][j];
    }
    __device__ __forceinline__ void clear(int k)
    {
#pragma unroll
        for (int j = 0; j < 8; ++j) at(k, j) = 0.0f;
    }
};

template <int DT, bool VEC, bool LAYER, bool BIAS, bool SHARED>
__global__ void __launch_bounds__(SHARED ? 1024 : 512) block_norm_grad_kernel(const __grid_constant__ NormParams P)
{
    __shared__ float area[2 * kSumArea];
    extern __shared__ float acc_shared[];
    constexpr int NACC = BIAS ? 5 : 3;
    const int T = blockDim.x;
    const Lane<VEC> L(threadIdx.x, T, P.dim);
    const int64_t worker = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int64_t r0 = worker * P.chunk, r1 = min(P.rows, r0 + P.chunk);
    if (r0 >= r1) return;                         // whole blocks, or warps that sum by themselves
    Acc<SHARED, NACC> acc(acc_shared, threadIdx.x, T);
    const Raw post_w = load_weight<DT, VEC>(P.post_w, L, 1.0f), post_b = load_weight<DT, VEC>(P.post_b, L, 0.0f);
    const Raw pre_w = load_weight<DT, VEC>(P.pre_w, L, 1.0f);
    const bool use_h = P.h != nullptr;
    int turn = 0;
    Raw h = {}, y = {}, dy = {}, dz = {}, gate = {};
    int64_t group = 0, group_first = 0;           // of the current row; the group's first row in the worker
    auto fetch = [&](int64_t r) {
        if (use_h) h = load_raw<VEC>(P.h + r * P.ld_h, L);
        if (P.pre) {
            y = load_raw<VEC>(P.y_in + r * P.ld_y, L);
            dz = load_raw<VEC>(P.dz + r * P.ld_dz, L);
        }
        if (P.dy) dy = load_raw<VEC>(P.dy + r * P.ld_dy, L);
    };
    fetch(r0);
    if (P.gate_rows) {
        group = r0 / P.gate_rows;
        group_first = r0;
        if (P.gate) gate = load_raw<VEC>(P.gate + group * P.ld_gate, L);
    }
    for (int64_t row = r0; row < r1; ++row) {
        float a[8], b[8], c[8], d[8], g[8], w[8];
        widen8<DT>(h, a);
        widen8<DT>(y, b);
        widen8<DT>(dz, c);
        widen8<DT>(dy, d);
        if (P.gate) widen8<DT>(gate, g);
        const int64_t this_group = group;
        if (row + 1 < r1) {
            fetch(row + 1);
            if (P.gate_rows) {
                group = (row + 1) / P.gate_rows;
                if (P.gate && group != this_group) gate = load_raw<VEC>(P.gate + group * P.ld_gate, L);
            }
        }
        // b, a: centred y and h; their sums, and those of g = dz w_pre
        widen8<DT>(pre_w, w);
        if constexpr (LAYER) {
            float s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s[0] += a[j];
                s[1] += b[j];
            }
            row_sum(s, T, area, turn);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (P.post) a[j] = j < L.n ? a[j] - s[0] * P.inv_dim : 0.0f;
                b[j] = j < L.n ? b[j] - s[1] * P.inv_dim : 0.0f;
            }
        }
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s[0] = fmaf(a[j], a[j], s[0]);
            s[1] = fmaf(b[j], b[j], s[1]);
            s[2] = fmaf(c[j] * w[j], b[j], s[2]);
            if (LAYER) s[3] = fmaf(c[j], w[j], s[3]);
        }
        if constexpr (LAYER) {
            row_sum(s, T, area, turn);
        } else {
            float t[3] = {s[0], s[1], s[2]};
            row_sum(t, T, area, turn);
            s[0] = t[0];
            s[1] = t[1];
            s[2] = t[2];
        }
        const float rh = rsqrtf(s[0] * P.inv_dim + P.eps), ry = rsqrtf(s[1] * P.inv_dim + P.eps);
        if (P.pre) {
            const float along = s[2] * P.inv_dim * ry * ry, mean = LAYER ? s[3] * P.inv_dim : 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                acc.at(kPreW, j) += c[j] * (b[j] * ry);
                if constexpr (BIAS) acc.at(kPreB, j) += c[j];
                d[j] += ry * (c[j] * w[j] - mean - b[j] * along);
            }
        }
        if (P.dx) store_row<DT, VEC>(P.dx + row * P.ld_dx, L, d);
        // through the gate: b becomes the normalised h, d becomes du
        if (P.post) {
            widen8<DT>(post_w, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) b[j] = a[j] * rh;
        }
        if (P.dgate) {
            float u[8];
            if (P.post) {
                widen8<DT>(post_b, u);
#pragma unroll
                for (int j = 0; j < 8; ++j) u[j] = fmaf(b[j], w[j], u[j]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) u[j] = a[j];
            }
            if (P.gate_rows == 1) {
#pragma unroll
                for (int j = 0; j < 8; ++j) u[j] = P.scale * d[j] * u[j];
                store_row<DT, VEC>(P.dgate + row * P.ld_dgate, L, u);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) acc.at(kGate, j) += P.scale * d[j] * u[j];
                if (row + 1 == r1 || group != this_group) {
                    // the end of the group, or of the worker: whole groups are final
                    const int64_t first = this_group * P.gate_rows, last = min(P.rows, first + P.gate_rows) - 1;
                    float t[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) t[j] = acc.at(kGate, j);
                    if (first >= r0 && last < r1) {
                        store_row<DT, VEC>(P.dgate + this_group * P.ld_dgate, L, t);
                    } else {
                        float* q = P.gate_sums + (worker * 2 + (group_first == r0 ? 0 : 1)) * P.dim;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (j < L.n) q[L.at(j)] = t[j];
                    }
                    acc.clear(kGate);
                    group_first = row + 1;
                }
            }
        }
        if (!P.dh && !P.sums) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] *= P.gate ? P.scale * g[j] : P.scale;
        if (P.post) {
            float t[2] = {0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                acc.at(kPostW, j) += d[j] * b[j];
                if constexpr (BIAS) acc.at(kPostB, j) += d[j];
                d[j] = j < L.n ? d[j] * w[j] : 0.0f;
                t[0] = fmaf(d[j], b[j], t[0]);
                t[1] += d[j];
            }
            if constexpr (LAYER) {
                row_sum(t, T, area, turn);
            } else {
                float one[1] = {t[0]};
                row_sum(one, T, area, turn);
                t[0] = one[0];
            }
            const float along = t[0] * P.inv_dim, mean = LAYER ? t[1] * P.inv_dim : 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] = rh * (d[j] - mean - b[j] * along);
        }
        if (P.dh) store_row<DT, VEC>(P.dh + row * P.ld_dh, L, d);
    }
    if (P.sums) {
        float* q = P.sums + worker * 4 * P.dim;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j < L.n) {
                const int e = L.at(j);
                q[e] = acc.at(kPreW, j);
                q[2 * P.dim + e] = acc.at(kPostW, j);
                if constexpr (BIAS) {
                    q[P.dim + e] = acc.at(kPreB, j);
                    q[3 * P.dim + e] = acc.at(kPostB, j);
                }
            }
        }
    }
}

struct SumParams {
    const float* sums;
    const float* gate_sums;
    uint16_t* out[4];          // dpre_w, dpre_b, dpost_w, dpost_b, or NULL
    uint16_t* dgate;
    int64_t rows, ld_dgate, gate_rows, chunk, workers;
    int32_t dim;
    int32_t by_group;          // gate sums: a block row a group, or a worker
};

// Block (column chunk, j): j < 4 adds the workers' sums of one weight; j >= 4 the parts of one gate
// group that spans workers.  32 columns by 32 workers at a time, in a fixed order.
template <int DT>
__global__ void __launch_bounds__(1024) block_norm_sum_kernel(const __grid_constant__ SumParams P)
{
    __shared__ float part[32][33];
    const int col = blockIdx.x * 32 + threadIdx.x, lane = threadIdx.y;
    float s = 0.0f;
    uint16_t* out;
    if (blockIdx.y < 4) {
        out = P.out[blockIdx.y];
        if (!out) return;
        if (col < P.dim)
            for (int64_t w = lane; w < P.workers; w += 32) s += P.sums[(w * 4 + blockIdx.y) * P.dim + col];
    } else {
        if (!P.dgate) return;
        const int64_t i = blockIdx.y - 4;
        const int64_t group = P.by_group ? i : (min(P.rows, (i + 1) * P.chunk) - 1) / P.gate_rows;
        const int64_t first = group * P.gate_rows, last = min(P.rows, first + P.gate_rows) - 1;
        const int64_t w0 = first / P.chunk, w1 = last / P.chunk;
        if (w0 == w1 || (!P.by_group && w0 != i)) return;      // whole in one worker, or another block's
        out = P.dgate + group * P.ld_dgate;
        if (col < P.dim)
            for (int64_t w = w0 + lane; w <= w1; w += 32)
                s += P.gate_sums[(w * 2 + (w == w0 && first > w0 * P.chunk ? 1 : 0)) * P.dim + col];
    }
    part[lane][threadIdx.x] = s;
    __syncthreads();
    if (lane == 0 && col < P.dim) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += part[i][threadIdx.x];
        out[col] = narrow1<DT>(s);
    }
}

// ------------------------------------------------------------------ host

constexpr int kSms = 152;

// Threads of a row, eight elements each; rows up to 256 elements are one warp, eight a block.
int row_threads(int64_t dim) { return std::max(32, (int)((dim + 7) / 8 + 31) / 32 * 32); }

// How the backward pass cuts the rows: workers of `chunk` consecutive ones.
struct Cut {
    int T = 32, per_block = 1;
    bool shared = false;
    int64_t chunk = 1, workers = 0;
};

Cut cut_rows(const zero_block_norm_t& a)
{
    Cut c;
    c.T = row_threads(a.dim);
    c.per_block = c.T == 32 ? 8 : 1;
    c.shared = c.T > 512;
    const int blocks_per_sm = std::max(1, 512 / (c.T * c.per_block));
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
    if (P.post) {
        P.post_w = in(a.post_w);
        P.post_b = in(a.post_b);
    }
    if (P.pre) {
        P.pre_w = in(a.pre_w);
        P.pre_b = in(a.pre_b);
    }
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

template <int DT, bool VEC, bool LAYER>
void launch_forward(const NormParams& P, cudaStream_t s)
{
    const int T = row_threads(P.dim), per_block = T == 32 ? 8 : 1;
    const int64_t blocks = (P.rows + per_block - 1) / per_block;
    const int64_t most = (int64_t)kSms * std::max(1, 1536 / (T * per_block));
    const unsigned grid = (unsigned)std::min(blocks, most);
    // registers are allotted for the largest block a kernel may have: rows beyond 4096 elements are apart
    if (T <= 512) block_norm_kernel<DT, VEC, LAYER, 512><<<grid, dim3(T, per_block), 0, s>>>(P);
    else block_norm_kernel<DT, VEC, LAYER, 1024><<<grid, dim3(T, per_block), 0, s>>>(P);
}

template <int DT, bool VEC, bool LAYER, bool BIAS>
zero_status_t launch_backward(const NormParams& P, const Cut& c, cudaStream_t s)
{
    const dim3 threads(c.T, c.per_block);
    const unsigned grid = (unsigned)((c.workers + c.per_block - 1) / c.per_block);
    if (c.shared) {
        constexpr int kMost = (BIAS ? 5 : 3) * 8 * 1024 * 4;
        static const cudaError_t set = cudaFuncSetAttribute(block_norm_grad_kernel<DT, VEC, LAYER, BIAS, true>,
                                                            cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
        if (set != cudaSuccess) return cuda_fail(set, "zero_block_norm_backward: shared memory");
        const int bytes = (BIAS ? 5 : 3) * 8 * c.T * 4;
        block_norm_grad_kernel<DT, VEC, LAYER, BIAS, true><<<grid, threads, bytes, s>>>(P);
    } else {
        block_norm_grad_kernel<DT, VEC, LAYER, BIAS, false><<<grid, threads, 0, s>>>(P);
    }
    return ZERO_OK;
}

template <int DT, bool VEC, bool LAYER>
zero_status_t launch_backward(const NormParams& P, const Cut& c, bool bias, cudaStream_t s)
{
    return bias ? launch_backward<DT, VEC, LAYER, true>(P, c, s) : launch_backward<DT, VEC, LAYER, false>(P, c, s);
}

template <int DT>
zero_status_t launch_backward(const NormParams& P, const Checked& C, bool bias, cudaStream_t s)
{
    const bool layer = C.a.kind == ZERO_NORM_LAYER;
    if (C.vec) return layer ? launch_backward<DT, true, true>(P, C.cut, bias, s) : launch_backward<DT, true, false>(P, C.cut, bias, s);
    return layer ? launch_backward<DT, false, true>(P, C.cut, bias, s) : launch_backward<DT, false, false>(P, C.cut, bias, s);
}

template <int DT>
void launch_forward(const NormParams& P, const Checked& C, cudaStream_t s)
{
    const bool layer = C.a.kind == ZERO_NORM_LAYER;
    if (C.vec) layer ? launch_forward<DT, true, true>(P, s) : launch_forward<DT, true, false>(P, s);
    else layer ? launch_forward<DT, false, true>(P, s) : launch_forward<DT, false, false>(P, s);
}

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" {

zero_status_t zero_block_norm(const zero_block_norm_t* args, void* stream)
try {
    Checked C;
    const zero_status_t st = check_norm(args, false, &C, "zero_block_norm");
    if (st != ZERO_OK) return st;
    if (C.a.rows == 0) return ZERO_OK;
    const NormParams P = params_of(C, false);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (C.a.dtype16 == ZERO_BF16) launch_forward<ZERO_BF16>(P, C, s);
    else launch_forward<ZERO_FP16>(P, C, s);
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
    const bool bias = a.dpre_b || a.dpost_b, bf = a.dtype16 == ZERO_BF16;
    if (a.rows > 0) {
        st = bf ? launch_backward<ZERO_BF16>(P, C, bias, s) : launch_backward<ZERO_FP16>(P, C, bias, s);
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
        const dim3 grid((unsigned)((a.dim + 31) / 32), (unsigned)(4 + (gates ? std::min(C.groups, C.cut.workers) : 0)));
        if (bf) block_norm_sum_kernel<ZERO_BF16><<<grid, dim3(32, 32), 0, s>>>(S);
        else block_norm_sum_kernel<ZERO_FP16><<<grid, dim3(32, 32), 0, s>>>(S);
    }
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "zero_block_norm_backward: launch");
}
catch (...) {
    return exception_status("zero_block_norm_backward");
}

}  // extern "C"
