// zero_adamw.cu -- one AdamW step over many separately held tensors (zero_adamw_*), first and
// second moments in 8 or 32 bits.
//
// The rule is the sharded step's (adamw1): every fp32 operation rounded by itself.  With 8-bit
// moments each block of 256 elements of one tensor keeps two power-of-two scales, so that scaling
// is exact and a stored moment is rounded once:
//   m         e4m3 times 2^(em - 127), em = max(1, exponent field of the block's largest |m| - 7)
//   sqrt(v)   an unsigned float of 4 exponent and 4 fraction bits (field 14 = [1, 2)) times
//             2^(er - 127), er = the exponent field of the block's largest sqrt(v); code 255 is
//             "not finite", and a root above 0 is never stored as 0 (an m that survived next to a
//             v that did not would make the next update m / eps)
// The root is kept instead of v because it is what the update divides by: 18 binades of it cover
// 36 of v, at half an ulp of 1/32.
//
// Bytes per element: gradient 2 or 4, fp32 parameter 4 + 4, 16-bit copy 2, moments 2 + 2 (8 bits) or
// 8 + 8 (32 bits): bound by HBM.  One warp takes one block of 256 elements, 8 to a lane in
// registers, so that the block's new maxima are two warp reductions and nothing is read twice.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <memory>
#include <vector>

#include <cuda_fp8.h>

#include "zero_device.cuh"

namespace zero {
namespace {

constexpr int kBlockElems = ZERO_ADAMW_BLOCK;  // elements of one tensor that share a pair of scales
constexpr int kAdamThreads = 256;
constexpr int kAdamWarps = kAdamThreads / 32;
constexpr int kAdamNormSlots = 4096;           // most blocks of a norm launch

// First 128 bytes of the workspace.
struct AdamState {
    int64_t t;            // applied steps
    int64_t skipped;      // skipped steps, total
    int64_t finished;
    double norm2;         // the running step's sum of squares (norm pass)
    double last_norm2;
    uint32_t flag;        // the norm pass met inf or nan
    uint32_t last_skipped;
    uint32_t last_norm_valid;
    uint32_t norm_tickets, step_tickets;   // blocks of the running launch that are done
    uint32_t pad;
};
static_assert(sizeof(AdamState) <= 128, "AdamState fits its slot");

// One tensor, as the kernels read it.
struct AdamTensor {
    float* p;
    uint16_t* p16;        // may be NULL
    const void* g;
    int64_t n;
    int32_t first;        // its first block
    int32_t vec;          // p, p16 and g start on 16 bytes
};
static_assert(sizeof(AdamTensor) == 40, "AdamTensor layout");

struct AdamParams {
    const AdamTensor* tensors;
    const int32_t* tensor_of;  // block -> tensor
    void* m;
    void* v;
    uint16_t* scales;          // 8 bits: low byte em, high byte er
    AdamState* st;
    double* partials;          // norm pass: one slot a launched block
    int32_t n_blocks;
    int32_t checked;           // a norm pass of this step ran: skip on its flag, clip by its norm
    float k[6];                // b1, 1-b1, b2, 1-b2, eps, lr*wd
    float inv;                 // 1 / loss scale
    double lr, beta1, beta2, max_norm;
};

// b^t in double by repeated squaring (t >= 0).
__device__ __forceinline__ double pow_int(double b, int64_t t)
{
    double r = 1.0;
    for (; t > 0; t >>= 1) {
        if (t & 1) r *= b;
        b *= b;
    }
    return r;
}

__device__ __forceinline__ float power_field(uint32_t e) { return __uint_as_float(e << 23); }

template <int GT>
__device__ __forceinline__ float load_grad1(const void* g, int64_t e)
{
    if constexpr (GT == ZERO_FP32) return static_cast<const float*>(g)[e];
    else return widen1<GT>(static_cast<const uint16_t*>(g)[e]);
}

// Eight gradients from element e on; aligned to 16 bytes.
template <int GT>
__device__ __forceinline__ void load_grad8(const void* g, int64_t e, float (&x)[8])
{
    if constexpr (GT == ZERO_FP32) {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(g) + e);
        const float4 a = __ldcs(q), b = __ldcs(q + 1);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
        const uint4 w = ld_stream(static_cast<const uint16_t*>(g) + e);
        widen2<GT>(w.x, x[0], x[1]);
        widen2<GT>(w.y, x[2], x[3]);
        widen2<GT>(w.z, x[4], x[5]);
        widen2<GT>(w.w, x[6], x[7]);
    }
}

// Which elements of its block a lane holds: eight in a row where the tensor's pointers allow
// 16-byte accesses, else every 32nd (32 lanes then touch neighbouring elements).
__device__ __forceinline__ int lane_elem(bool vec, int lane, int j) { return vec ? lane * 8 + j : j * 32 + lane; }

// ---------------------------------------------------------------- 8-bit moments

__device__ __forceinline__ void decode_m8(uint2 c, float scale, float (&m)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_fp8x2_storage_t q = (__nv_fp8x2_storage_t)((i < 2 ? c.x : c.y) >> (16 * (i & 1)));
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(q, __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        m[2 * i] = __fmul_rn(f.x, scale);
        m[2 * i + 1] = __fmul_rn(f.y, scale);
    }
}

__device__ __forceinline__ uint2 encode_m8(const float (&m)[8], float inv)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(m[2 * i], inv), __fmul_rn(m[2 * i + 1], inv)),
                                        __NV_SATFINITE, __NV_E4M3);
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// A code's value: its bits moved to a float's exponent and fraction are the value times 2^-113
// (field 0 becomes a subnormal, as it should), so one exact product gives it.
__device__ __forceinline__ float decode_root1(uint32_t c, float scale)
{
    const float y = __fmul_rn(__uint_as_float(c << 19), power_field(127 + 113));
    return c == 255u ? __uint_as_float(0x7FC00000u) : __fmul_rn(y, scale);
}

__device__ __forceinline__ uint32_t encode_root1(float r, float inv)
{
    const float y = __fmul_rn(r, inv);                       // in [0, 2)
    const uint32_t b = __float_as_uint(y);
    uint32_t c = ((b + 0x3FFFFu + ((b >> 19) & 1u)) >> 19) - (113u << 4);
    if (y < 0x1p-13f) c = (uint32_t)__float2int_rn(__fmul_rn(y, 0x1p17f));
    if (c == 0u && y > 0.0f) c = 1u;
    return min(c, 255u);
}

// Largest exponent field of eight magnitudes over the warp; of the finite ones where some are not.
__device__ __forceinline__ uint32_t warp_top_field(const float (&x)[8])
{
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (top >= 0x7F800000u) {
        top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (!nonfinite(x[j])) top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
        top = __reduce_max_sync(0xFFFFFFFFu, top);
    }
    return top >> 23;
}

// ---------------------------------------------------------------- kernels

template <int BITS, int GT, int DT>
__global__ void __launch_bounds__(kAdamThreads) adamw_kernel(const __grid_constant__ AdamParams P)
{
    __shared__ float sk_shared[4];
    __shared__ bool skip;
    const int lane = threadIdx.x & 31;
    // the constants of this step: two lanes raise the betas to the step's power
    if (threadIdx.x < 32) {
        const volatile AdamState* st = P.st;
        const int64_t t = st->t + 1;
        const double bc = 1.0 - pow_int(lane == 0 ? P.beta1 : P.beta2, t);
        if (lane == 0) {
            sk_shared[0] = __double2float_rn(__ddiv_rn(P.lr, bc));
            sk_shared[3] = 1.0f;
            bool s = false;
            if (P.checked) {
                s = st->flag != 0;
                if (P.max_norm > 0.0) {
                    const double c = __ddiv_rn(P.max_norm, __dadd_rn(__dsqrt_rn(st->norm2), 1e-6));
                    sk_shared[3] = __double2float_rn(c > 1.0 ? 1.0 : c);
                }
            }
            skip = s;
        } else if (lane == 1) {
            sk_shared[1] = __double2float_rn(__dsqrt_rn(bc));
        }
    }
    __syncthreads();
    StepK sk;
    sk.step = sk_shared[0];
    sk.bc2s = sk_shared[1];
    sk.inv = P.inv;
    sk.coef = sk_shared[3];

    const int stride = gridDim.x * kAdamWarps;
    if (!skip) {
        for (int b = blockIdx.x * kAdamWarps + (threadIdx.x >> 5); b < P.n_blocks; b += stride) {
            const AdamTensor T = P.tensors[__ldg(P.tensor_of + b)];
            const int64_t e0 = (int64_t)(b - T.first) * kBlockElems;      // in the tensor
            const int64_t s0 = (int64_t)b * kBlockElems;                  // in the moments
            const int n = (int)min((int64_t)kBlockElems, T.n - e0);
            // whole groups of eight only; the lane that holds the tensor's end goes by element
            const bool vec = T.vec != 0;
            const bool full = vec && lane * 8 + 8 <= n;
            float g[8], p[8], m[8], v[8];
            if (full) {
                load_grad8<GT>(T.g, e0 + lane * 8, g);
                const float4* q = reinterpret_cast<const float4*>(T.p + e0 + lane * 8);
                const float4 a = __ldcs(q), c = __ldcs(q + 1);
                p[0] = a.x; p[1] = a.y; p[2] = a.z; p[3] = a.w;
                p[4] = c.x; p[5] = c.y; p[6] = c.z; p[7] = c.w;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int e = lane_elem(vec, lane, j);
                    g[j] = e < n ? load_grad1<GT>(T.g, e0 + e) : 0.0f;
                    p[j] = e < n ? T.p[e0 + e] : 0.0f;
                }
            }
            // the moments' block is padded to 256 elements and starts on 16 bytes
            if constexpr (BITS == 32) {
                float* mp = static_cast<float*>(P.m) + s0;
                float* vp = static_cast<float*>(P.v) + s0;
                if (vec) {
                    const float4 a = __ldcs(reinterpret_cast<const float4*>(mp + lane * 8));
                    const float4 c = __ldcs(reinterpret_cast<const float4*>(mp + lane * 8) + 1);
                    const float4 d = __ldcs(reinterpret_cast<const float4*>(vp + lane * 8));
                    const float4 f = __ldcs(reinterpret_cast<const float4*>(vp + lane * 8) + 1);
                    m[0] = a.x; m[1] = a.y; m[2] = a.z; m[3] = a.w;
                    m[4] = c.x; m[5] = c.y; m[6] = c.z; m[7] = c.w;
                    v[0] = d.x; v[1] = d.y; v[2] = d.z; v[3] = d.w;
                    v[4] = f.x; v[5] = f.y; v[6] = f.z; v[7] = f.w;
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        m[j] = mp[j * 32 + lane];
                        v[j] = vp[j * 32 + lane];
                    }
                }
            } else {
                const uint8_t* mp = static_cast<const uint8_t*>(P.m) + s0;
                const uint8_t* vp = static_cast<const uint8_t*>(P.v) + s0;
                uint2 mc, vc;
                if (vec) {
                    mc = __ldcs(reinterpret_cast<const uint2*>(mp + lane * 8));
                    vc = __ldcs(reinterpret_cast<const uint2*>(vp + lane * 8));
                } else {
                    mc = vc = make_uint2(0u, 0u);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t a = mp[j * 32 + lane], c = vp[j * 32 + lane];
                        if (j < 4) {
                            mc.x |= a << (8 * j);
                            vc.x |= c << (8 * j);
                        } else {
                            mc.y |= a << (8 * (j - 4));
                            vc.y |= c << (8 * (j - 4));
                        }
                    }
                }
                const uint32_t e = P.scales[b];
                decode_m8(mc, power_field(e & 0xFFu), m);
                const float rs = power_field(e >> 8);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float r = decode_root1(((j < 4 ? vc.x : vc.y) >> (8 * (j & 3))) & 0xFFu, rs);
                    v[j] = __fmul_rn(r, r);
                }
            }
            float root[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float gu = __fmul_rn(__fmul_rn(g[j], sk.inv), sk.coef);
                m[j] = __fadd_rn(__fmul_rn(P.k[0], m[j]), __fmul_rn(P.k[1], gu));
                v[j] = __fadd_rn(__fmul_rn(P.k[2], v[j]), __fmul_rn(P.k[3], __fmul_rn(gu, gu)));
                root[j] = __fsqrt_rn(v[j]);
                const float d = __fadd_rn(__fdiv_rn(root[j], sk.bc2s), P.k[4]);
                p[j] = __fsub_rn(p[j], __fmul_rn(P.k[5], p[j]));
                p[j] = __fsub_rn(p[j], __fmul_rn(sk.step, __fdiv_rn(m[j], d)));
            }
            if (full) {
                float4* q = reinterpret_cast<float4*>(T.p + e0 + lane * 8);
                __stcs(q, make_float4(p[0], p[1], p[2], p[3]));
                __stcs(q + 1, make_float4(p[4], p[5], p[6], p[7]));
                if (T.p16)
                    __stcs(reinterpret_cast<uint4*>(T.p16 + e0 + lane * 8),
                           make_uint4(narrow2<DT>(p[0], p[1]), narrow2<DT>(p[2], p[3]),
                                      narrow2<DT>(p[4], p[5]), narrow2<DT>(p[6], p[7])));
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int e = lane_elem(vec, lane, j);
                    if (e < n) {
                        T.p[e0 + e] = p[j];
                        if (T.p16) T.p16[e0 + e] = narrow1<DT>(p[j]);
                    } else {
                        m[j] = v[j] = root[j] = 0.0f;      // the moments' padding stays zero
                    }
                }
            }
            if constexpr (BITS == 32) {
                float* mp = static_cast<float*>(P.m) + s0;
                float* vp = static_cast<float*>(P.v) + s0;
                if (vec) {
                    float4* a = reinterpret_cast<float4*>(mp + lane * 8);
                    float4* c = reinterpret_cast<float4*>(vp + lane * 8);
                    __stcs(a, make_float4(m[0], m[1], m[2], m[3]));
                    __stcs(a + 1, make_float4(m[4], m[5], m[6], m[7]));
                    __stcs(c, make_float4(v[0], v[1], v[2], v[3]));
                    __stcs(c + 1, make_float4(v[4], v[5], v[6], v[7]));
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        mp[j * 32 + lane] = m[j];
                        vp[j * 32 + lane] = v[j];
                    }
                }
            } else {
                // an infinite m would saturate to a finite code: it is kept as not a number
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (nonfinite(m[j])) m[j] = __uint_as_float(0x7FC00000u);
                const uint32_t fm = warp_top_field(m), er = warp_top_field(root);
                const uint32_t em = fm > 8u ? fm - 7u : 1u;
                const uint2 mc = encode_m8(m, power_field(254u - em));
                const float ri = power_field(254u - er);
                uint2 vc = make_uint2(0u, 0u);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    vc.x |= encode_root1(root[j], ri) << (8 * j);
                    vc.y |= encode_root1(root[j + 4], ri) << (8 * j);
                }
                uint8_t* mp = static_cast<uint8_t*>(P.m) + s0;
                uint8_t* vp = static_cast<uint8_t*>(P.v) + s0;
                if (vec) {
                    __stcs(reinterpret_cast<uint2*>(mp + lane * 8), mc);
                    __stcs(reinterpret_cast<uint2*>(vp + lane * 8), vc);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        mp[j * 32 + lane] = (uint8_t)((j < 4 ? mc.x : mc.y) >> (8 * (j & 3)));
                        vp[j * 32 + lane] = (uint8_t)((j < 4 ? vc.x : vc.y) >> (8 * (j & 3)));
                    }
                }
                if (lane == 0) P.scales[b] = (uint16_t)(em | (er << 8));
            }
        }
    }
    // the last block to finish closes the step: every block has read t by then
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        if (atomicAdd(&P.st->step_tickets, 1u) == gridDim.x - 1) {
            volatile AdamState* st = P.st;
            st->step_tickets = 0;
            st->finished = st->finished + 1;
            if (skip) st->skipped = st->skipped + 1;
            else st->t = st->t + 1;
            st->last_skipped = skip ? 1u : 0u;
            st->last_norm_valid = P.checked ? 1u : 0u;
            st->last_norm2 = P.checked ? st->norm2 : 0.0;
        }
    }
}

// The sum of squares of the unscaled gradient and whether all of it is finite.  The order of the
// sum is fixed: lanes, then warps, then blocks in order.
template <int GT>
__global__ void __launch_bounds__(kAdamThreads) adamw_norm_kernel(const __grid_constant__ AdamParams P)
{
    __shared__ double warp_sum[kAdamWarps];
    __shared__ bool last;
    __shared__ uint32_t any_bad;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) any_bad = 0;
    NormAcc acc;
    bool bad = false;
    const int stride = gridDim.x * kAdamWarps;
    for (int b = blockIdx.x * kAdamWarps + (threadIdx.x >> 5); b < P.n_blocks; b += stride) {
        const AdamTensor T = P.tensors[__ldg(P.tensor_of + b)];
        const int64_t e0 = (int64_t)(b - T.first) * kBlockElems;
        const int n = (int)min((int64_t)kBlockElems, T.n - e0);
        const bool vec = T.vec != 0;
        float g[8];
        if (vec && lane * 8 + 8 <= n) {
            load_grad8<GT>(T.g, e0 + lane * 8, g);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int e = lane_elem(vec, lane, j);
                g[j] = e < n ? load_grad1<GT>(T.g, e0 + e) : 0.0f;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = __fmul_rn(g[j], P.inv);
            bad |= nonfinite(x);
            acc.add(__fmul_rn(x, x));
        }
    }
    __syncthreads();
    if (bad) any_bad = 1;
    const double s = block_sum_fixed<kAdamThreads>(acc.value(), warp_sum);
    if (threadIdx.x == 0) {
        // a block's slot holds its sum, or not-a-number as the mark of a gradient that is not finite
        P.partials[blockIdx.x] = any_bad ? __longlong_as_double(0x7FF8000000000000ll) : s;
        __threadfence();
        last = atomicAdd(&P.st->norm_tickets, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    const volatile double* slots = P.partials;
    double x = 0.0;
    for (unsigned i = threadIdx.x; i < gridDim.x; i += kAdamThreads) x += slots[i];
    const double sum = block_sum_fixed<kAdamThreads>(x, warp_sum);
    if (threadIdx.x == 0) {
        volatile AdamState* st = P.st;
        st->norm2 = sum;
        st->flag = isnan(sum) ? 1u : 0u;
        st->norm_tickets = 0;
    }
}

// The 8-bit moments as the values that they stand for; bf16 holds each of them exactly.
__global__ void __launch_bounds__(kAdamThreads) adamw_export_kernel(const uint8_t* m, const uint8_t* v,
                                                                    const uint16_t* scales, uint16_t* m_out,
                                                                    uint16_t* root_out, int n_blocks)
{
    const int lane = threadIdx.x & 31, stride = gridDim.x * kAdamWarps;
    for (int b = blockIdx.x * kAdamWarps + (threadIdx.x >> 5); b < n_blocks; b += stride) {
        const int64_t at = (int64_t)b * kBlockElems + lane * 8;
        const uint2 mc = __ldcs(reinterpret_cast<const uint2*>(m + at));
        const uint2 vc = __ldcs(reinterpret_cast<const uint2*>(v + at));
        const uint32_t e = scales[b];
        float x[8], r[8];
        decode_m8(mc, power_field(e & 0xFFu), x);
        const float rs = power_field(e >> 8);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = decode_root1(((j < 4 ? vc.x : vc.y) >> (8 * (j & 3))) & 0xFFu, rs);
        __stcs(reinterpret_cast<uint4*>(m_out + at),
               make_uint4(narrow2<ZERO_BF16>(x[0], x[1]), narrow2<ZERO_BF16>(x[2], x[3]),
                          narrow2<ZERO_BF16>(x[4], x[5]), narrow2<ZERO_BF16>(x[6], x[7])));
        __stcs(reinterpret_cast<uint4*>(root_out + at),
               make_uint4(narrow2<ZERO_BF16>(r[0], r[1]), narrow2<ZERO_BF16>(r[2], r[3]),
                          narrow2<ZERO_BF16>(r[4], r[5]), narrow2<ZERO_BF16>(r[6], r[7])));
    }
}

}  // namespace
}  // namespace zero

struct zero_adamw {
    int bits = 0, dtype16 = 0, grad_type = 0;
    std::vector<int64_t> sizes;
    int64_t elems = 0, n_blocks = 0;
    // bound buffers (caller-owned)
    bool bound = false;
    int device = -1;
    void *m = nullptr, *v = nullptr, *scales = nullptr, *workspace = nullptr;
};

namespace zero {
namespace {

// Workspace: the state's slot, the tensors, the blocks' tensors, the norm pass's slots.
constexpr int64_t kAdamStateBytes = 256;
inline int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }
int64_t tensors_at() { return kAdamStateBytes; }
int64_t map_at(const zero_adamw* h) { return tensors_at() + up16((int64_t)sizeof(AdamTensor) * (int64_t)h->sizes.size()); }
int64_t slots_at(const zero_adamw* h) { return map_at(h) + up16(4 * h->n_blocks); }
int64_t adam_workspace(const zero_adamw* h) { return slots_at(h) + 8 * kAdamNormSlots; }

// A persistent grid: as many blocks as fit the GPU at once, or as the work needs.
template <auto KERNEL>
int adam_grid(const zero_adamw* h)
{
    static const int per_sm = [] {
        int n = 0;
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, KERNEL, kAdamThreads, 0) == cudaSuccess ? std::max(1, n) : 1;
    }();
    const int64_t cap = (int64_t)std::max(1, device_sms(h->device)) * per_sm;
    const int64_t need = (h->n_blocks + kAdamWarps - 1) / kAdamWarps;
    return (int)std::max<int64_t>(1, std::min({cap, need, (int64_t)kAdamNormSlots}));
}

template <int BITS, int GT>
void launch_adamw(const zero_adamw* h, const AdamParams& P, cudaStream_t s)
{
    if (h->dtype16 == ZERO_BF16)
        adamw_kernel<BITS, GT, ZERO_BF16><<<adam_grid<adamw_kernel<BITS, GT, ZERO_BF16>>(h), kAdamThreads, 0, s>>>(P);
    else
        adamw_kernel<BITS, GT, ZERO_FP16><<<adam_grid<adamw_kernel<BITS, GT, ZERO_FP16>>(h), kAdamThreads, 0, s>>>(P);
}

template <int BITS>
void launch_adamw(const zero_adamw* h, const AdamParams& P, cudaStream_t s)
{
    if (h->grad_type == ZERO_BF16) launch_adamw<BITS, ZERO_BF16>(h, P, s);
    else if (h->grad_type == ZERO_FP16) launch_adamw<BITS, ZERO_FP16>(h, P, s);
    else launch_adamw<BITS, ZERO_FP32>(h, P, s);
}

template <int GT>
void launch_norm(const zero_adamw* h, const AdamParams& P, cudaStream_t s)
{
    adamw_norm_kernel<GT><<<adam_grid<adamw_norm_kernel<GT>>(h), kAdamThreads, 0, s>>>(P);
}

// The bound device has to be current: the launches go to it.
zero_status_t adam_ready(const zero_adamw* h, const char* who)
{
    if (!h) return fail(ZERO_EINVAL, std::string(who) + ": NULL handle");
    if (!h->bound) return fail(ZERO_ESTATE, std::string(who) + ": nothing bound (zero_adamw_bind)");
    int dev = -1;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, who);
    if (dev != h->device) return fail(ZERO_EINVAL, std::string(who) + ": the bound buffers live on another device");
    return ZERO_OK;
}

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" {

zero_status_t zero_adamw_create(const int64_t* tensor_sizes, int64_t n_tensors, int state_bits, int dtype16,
                                int grad_type, zero_adamw_t** out)
try {
    if (!out || (!tensor_sizes && n_tensors > 0)) return fail(ZERO_EINVAL, "zero_adamw_create: NULL argument");
    *out = nullptr;
    if (n_tensors < 0) return fail(ZERO_EINVAL, "zero_adamw_create: negative tensor count");
    if (state_bits != 8 && state_bits != 32) return fail(ZERO_EINVAL, "zero_adamw_create: state_bits must be 8 or 32");
    if (dtype16 != ZERO_BF16 && dtype16 != ZERO_FP16) return fail(ZERO_EINVAL, "zero_adamw_create: bad dtype16");
    if (grad_type != ZERO_BF16 && grad_type != ZERO_FP16 && grad_type != ZERO_FP32)
        return fail(ZERO_EINVAL, "zero_adamw_create: bad grad_type");
    std::unique_ptr<zero_adamw> h(new zero_adamw);
    h->bits = state_bits;
    h->dtype16 = dtype16;
    h->grad_type = grad_type;
    h->sizes.assign(tensor_sizes, tensor_sizes + n_tensors);
    for (const int64_t n : h->sizes) {
        if (n < 0) return fail(ZERO_EINVAL, "zero_adamw_create: negative tensor size");
        if (n > (int64_t)1 << 40) return fail(ZERO_ERANGE, "zero_adamw_create: a tensor beyond 2^40 elements");
        h->elems += n;
        h->n_blocks += (n + kBlockElems - 1) / kBlockElems;
        if (h->n_blocks > ZERO_ADAMW_MAX_BLOCKS)
            return fail(ZERO_ERANGE, "zero_adamw_create: more than ZERO_ADAMW_MAX_BLOCKS blocks");
    }
    if (n_tensors > INT32_MAX) return fail(ZERO_ERANGE, "zero_adamw_create: too many tensors");
    *out = h.release();
    return ZERO_OK;
}
catch (...) {
    return exception_status("zero_adamw_create");
}

zero_status_t zero_adamw_info(const zero_adamw_t* h, zero_adamw_info_t* out)
try {
    if (!h || !out) return fail(ZERO_EINVAL, "zero_adamw_info: NULL argument");
    out->n_tensors = (int64_t)h->sizes.size();
    out->elems = h->elems;
    out->n_blocks = h->n_blocks;
    out->state_elems = h->n_blocks * kBlockElems;
    out->moment_bytes = out->state_elems * (h->bits / 8);
    out->scale_bytes = h->bits == 8 ? 2 * h->n_blocks : 0;
    out->workspace_bytes = adam_workspace(h);
    return ZERO_OK;
}
catch (...) {
    return exception_status("zero_adamw_info");
}

zero_status_t zero_adamw_bind(zero_adamw_t* h, float* const* params, void* const* params16, const void* const* grads,
                              void* m, void* v, void* scales, void* workspace, int64_t t, void* stream)
try {
    if (!h) return fail(ZERO_EINVAL, "zero_adamw_bind: NULL handle");
    const size_t n = h->sizes.size();
    if (n > 0 && (!params || !grads)) return fail(ZERO_EINVAL, "zero_adamw_bind: NULL argument");
    if (!workspace) return fail(ZERO_EINVAL, "zero_adamw_bind: workspace is NULL");
    if (t < -1 || (t == -1 && !h->bound))
        return fail(ZERO_EINVAL, "zero_adamw_bind: t must be >= 0 (-1 keeps an earlier bind's)");
    if (t == -1 && workspace != h->workspace)
        return fail(ZERO_EINVAL, "zero_adamw_bind: t = -1 needs the earlier bind's workspace");
    if (h->n_blocks > 0) {
        if (!m || !v) return fail(ZERO_EINVAL, "zero_adamw_bind: NULL moments");
        if (h->bits == 8 && !scales) return fail(ZERO_EINVAL, "zero_adamw_bind: 8-bit moments need scales");
    }
    if (!aligned(m, 16) || !aligned(v, 16)) return fail(ZERO_EALIGN, "zero_adamw_bind: moments not 16-byte aligned");
    if (!aligned(scales, 2)) return fail(ZERO_EALIGN, "zero_adamw_bind: scales not 2-byte aligned");
    if (!aligned(workspace, 16)) return fail(ZERO_EALIGN, "zero_adamw_bind: workspace not 16-byte aligned");
    std::vector<unsigned char> image((size_t)(slots_at(h)), 0);
    AdamTensor* T = reinterpret_cast<AdamTensor*>(image.data() + tensors_at());
    int32_t* map = reinterpret_cast<int32_t*>(image.data() + map_at(h));
    const uintptr_t gsize = h->grad_type == ZERO_FP32 ? 4 : 2;
    int64_t block = 0;
    for (size_t i = 0; i < n; ++i) {
        const int64_t elems = h->sizes[i];
        if (elems > 0 && (!params[i] || !grads[i])) return fail(ZERO_EINVAL, "zero_adamw_bind: NULL tensor pointer");
        T[i].p = params[i];
        T[i].p16 = params16 ? static_cast<uint16_t*>(params16[i]) : nullptr;
        T[i].g = grads[i];
        T[i].n = elems;
        T[i].first = (int32_t)block;
        if (!aligned(T[i].p, 4) || !aligned(T[i].p16, 2) || !aligned(T[i].g, gsize))
            return fail(ZERO_EALIGN, "zero_adamw_bind: a tensor is not aligned to its element size");
        T[i].vec = aligned(T[i].p, 16) && aligned(T[i].p16, 16) && aligned(T[i].g, 16);
        const int64_t blocks = (elems + kBlockElems - 1) / kBlockElems;
        std::fill(map + block, map + block + blocks, (int32_t)i);
        block += blocks;
    }
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "zero_adamw_bind: cudaGetDevice");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    AdamState init;
    std::memset(&init, 0, sizeof(init));
    init.t = t;
    std::memcpy(image.data(), &init, sizeof(init));
    const size_t skip = t == -1 ? (size_t)tensors_at() : 0;       // -1: the state's slot stays
    e = cudaMemcpyAsync(static_cast<char*>(workspace) + skip, image.data() + skip, image.size() - skip,
                        cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e, "zero_adamw_bind: the workspace's tables");
    h->m = m;
    h->v = v;
    h->scales = scales;
    h->workspace = workspace;
    h->device = dev;
    h->bound = true;
    return ZERO_OK;
}
catch (...) {
    return exception_status("zero_adamw_bind");
}

zero_status_t zero_adamw_step(zero_adamw_t* h, const zero_hyper_t* hyper, double loss_scale, void* stream)
try {
    if (!h || !hyper) return fail(ZERO_EINVAL, "zero_adamw_step: NULL argument");
    if (!(hyper->beta1 >= 0.0 && hyper->beta1 < 1.0) || !(hyper->beta2 >= 0.0 && hyper->beta2 < 1.0))
        return fail(ZERO_EINVAL, "zero_adamw_step: betas must be in [0, 1)");
    if (!(hyper->eps >= 0.0) || !(hyper->max_grad_norm >= 0.0) || !std::isfinite(hyper->lr) ||
        !std::isfinite(hyper->weight_decay))
        return fail(ZERO_EINVAL, "zero_adamw_step: bad hyperparameter");
    if (hyper->flags & ~(int64_t)ZERO_REPORT_GRAD_NORM) return fail(ZERO_EINVAL, "zero_adamw_step: unknown flag");
    if (!(loss_scale > 0.0) || !std::isfinite(loss_scale))
        return fail(ZERO_EINVAL, "zero_adamw_step: loss_scale must be positive");
    const zero_status_t ready = adam_ready(h, "zero_adamw_step");
    if (ready != ZERO_OK) return ready;
    char* ws = static_cast<char*>(h->workspace);
    AdamParams P;
    float c[9];
    step_constants(*hyper, 1, loss_scale, 1, c);
    P.tensors = reinterpret_cast<const AdamTensor*>(ws + tensors_at());
    P.tensor_of = reinterpret_cast<const int32_t*>(ws + map_at(h));
    P.m = h->m;
    P.v = h->v;
    P.scales = static_cast<uint16_t*>(h->scales);
    P.st = reinterpret_cast<AdamState*>(ws);
    P.partials = reinterpret_cast<double*>(ws + slots_at(h));
    P.n_blocks = (int32_t)h->n_blocks;
    P.checked = hyper->max_grad_norm > 0.0 || (hyper->flags & ZERO_REPORT_GRAD_NORM);
    for (int i = 0; i < 6; ++i) P.k[i] = c[i];
    P.inv = c[8];
    P.lr = hyper->lr;
    P.beta1 = hyper->beta1;
    P.beta2 = hyper->beta2;
    P.max_norm = hyper->max_grad_norm;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (P.checked) {
        if (h->grad_type == ZERO_BF16) launch_norm<ZERO_BF16>(h, P, s);
        else if (h->grad_type == ZERO_FP16) launch_norm<ZERO_FP16>(h, P, s);
        else launch_norm<ZERO_FP32>(h, P, s);
    }
    if (h->bits == 8) launch_adamw<8>(h, P, s);
    else launch_adamw<32>(h, P, s);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "zero_adamw_step: launch");
}
catch (...) {
    return exception_status("zero_adamw_step");
}

zero_status_t zero_adamw_export(zero_adamw_t* h, void* m_out, void* root_out, void* stream)
try {
    if (!h || !m_out || !root_out) return fail(ZERO_EINVAL, "zero_adamw_export: NULL argument");
    if (h->bits != 8) return fail(ZERO_EINVAL, "zero_adamw_export: the moments are plain fp32 buffers");
    if (!aligned(m_out, 16) || !aligned(root_out, 16))
        return fail(ZERO_EALIGN, "zero_adamw_export: outputs not 16-byte aligned");
    const zero_status_t ready = adam_ready(h, "zero_adamw_export");
    if (ready != ZERO_OK) return ready;
    if (h->n_blocks == 0) return ZERO_OK;
    adamw_export_kernel<<<adam_grid<adamw_export_kernel>(h), kAdamThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint8_t*>(h->m), static_cast<const uint8_t*>(h->v), static_cast<const uint16_t*>(h->scales),
        static_cast<uint16_t*>(m_out), static_cast<uint16_t*>(root_out), (int)h->n_blocks);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "zero_adamw_export: launch");
}
catch (...) {
    return exception_status("zero_adamw_export");
}

zero_status_t zero_adamw_read(zero_adamw_t* h, void* stream, zero_step_result_t* out)
try {
    if (!h || !out) return fail(ZERO_EINVAL, "zero_adamw_read: NULL argument");
    const zero_status_t ready = adam_ready(h, "zero_adamw_read");
    if (ready != ZERO_OK) return ready;
    AdamState st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemcpyAsync(&st, h->workspace, sizeof(st), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e, "zero_adamw_read");
    std::memset(out, 0, sizeof(*out));
    out->skipped = (int32_t)st.last_skipped;
    out->t = st.t;
    out->scale = 1.0;
    out->good_steps = st.t;
    out->skipped_total = st.skipped;
    out->finished = st.finished;
    out->grad_norm = st.last_norm_valid ? std::sqrt(st.last_norm2) : -1.0;
    return ZERO_OK;
}
catch (...) {
    return exception_status("zero_adamw_read");
}

void zero_adamw_destroy(zero_adamw_t* h) { delete h; }

}  // extern "C"
