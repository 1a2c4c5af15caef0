// zero_adamw.cu -- one AdamW step over many separately held tensors (zero_adamw_*), first and
// second moments in 8 or 32 bits.
//
// The rule is the sharded step's: the moments' operations are each rounded by themselves (their codes
// hang on a last place, see below), the step's root and quotient are within 2 units in the last place.
// With 8-bit moments each block of 256 elements of one tensor keeps two power-of-two scales, so that
// scaling is exact and a stored moment is rounded once:
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
// Measured on one GB300, a step after another: 124M elements, fp16 gradients, 8 bits 362 us (5.5 TB/s of the
// 16 bytes an element), 59M elements, fp32 gradients, 32 bits 283 us (6.3 TB/s); 59M elements in 10,000
// packed tensors, 8 bits, clipped, with the values' export: 316 us, of which 44 are the norm, 219 the step and
// 56 the export.  adamw_export (6 bytes an element): 112 us of 124M.  194 gains and biases: 10 us a call.
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
constexpr int kAhead = 2;                       // 8-bit moments: blocks on their way to a warp
constexpr int kAdamPerSm8 = 2;
constexpr int kAdamPerSm32 = 3;
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

// One tensor, as bound.
struct AdamTensor {
    float* p;
    uint16_t* p16;        // may be NULL
    const void* g;
    int64_t n;
    int32_t first;        // its first block
    int32_t vec;          // p, p16 and g start on 16 bytes
};
static_assert(sizeof(AdamTensor) == 40, "AdamTensor layout");

// How a block's g, p and 16-bit copy are accessed.  kAligned: it is whole and they start on 16 bytes.
// kInner: it is whole and neither the tensor's first nor its last, so that the 4-byte words around its
// ends are the tensor's too.  kSingly: element by element.
enum { kSingly = 0, kAligned = 1, kInner = 2 };

// One block of a tensor, as the kernels read it: 32 bytes for the 4 KB and more that the block moves.
// (A table of tensors and one from blocks to tensors are smaller, but two reads one after the other.)
struct alignas(16) AdamBlock {
    float* p;             // at the block's first element
    uint16_t* p16;
    const void* g;
    int32_t n;            // elements, 1 .. kBlockElems
    int32_t vec;          // kAligned, kInner or kSingly
};
static_assert(sizeof(AdamBlock) == 32, "AdamBlock layout");

struct AdamParams {
    const AdamBlock* blocks;
    void* m;
    void* v;
    uint16_t* scales;          // 8 bits: low byte em, high byte er
    AdamState* st;
    double* partials;          // norm pass: one slot a launched block
    int32_t n_blocks;
    int32_t checked;           // a norm pass of this step ran: skip on its flag, clip by its norm
    DevState* plan;            // a sharded step that this one belongs to: skip on its flag, clip by its
                               // norm, unscale by its loss scale; or NULL
    F2 k[6];                   // b1, 1-b1, b2, 1-b2, eps, -lr*wd, each twice
    F2 one;                    // 1 (add_apart)
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

// ---------------------------------------------------------------- a warp's block of one tensor

// Which elements of its block a lane holds: four in a row from 4 lane on, and four from 128 + 4 lane on, so
// that 32 lanes' 16-byte accesses to fp32 values cover 512 bytes without gaps (eight in a row leave half
// of every sector to a second access).  In a kSingly block every 32nd.

// The table is constant for a kernel's lifetime: zero_adamw_bind waits for the kernel that writes it.
__device__ __forceinline__ AdamBlock block_at(const AdamParams& P, int b)
{
    AdamBlock B;
    const uint4* q = reinterpret_cast<const uint4*>(P.blocks + b);
    reinterpret_cast<uint4*>(&B)[0] = __ldg(q);
    reinterpret_cast<uint4*>(&B)[1] = __ldg(q + 1);
    return B;
}

template <int GT>
__device__ __forceinline__ float load_grad1(const void* g, int64_t e)
{
    if constexpr (GT == ZERO_FP32) return static_cast<const float*>(g)[e];
    else return widen1<GT>(static_cast<const uint16_t*>(g)[e]);
}

template <int GT>
__device__ __forceinline__ void load_grads(const AdamBlock& B, int lane, float (&x)[8])
{
    if (B.vec == kAligned) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (GT == ZERO_FP32) {
                const float4 q = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(B.g) + i * 128 + lane * 4));
                x[4 * i] = q.x; x[4 * i + 1] = q.y; x[4 * i + 2] = q.z; x[4 * i + 3] = q.w;
            } else {
                const uint2 q = ld_stream8(static_cast<const uint16_t*>(B.g) + i * 128 + lane * 4);
                widen2<GT>(q.x, x[4 * i], x[4 * i + 1]);
                widen2<GT>(q.y, x[4 * i + 2], x[4 * i + 3]);
            }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = j * 32 + lane < B.n ? load_grad1<GT>(B.g, j * 32 + lane) : 0.0f;
}

// A lane's eight of 256 consecutive fp32 values.
__device__ __forceinline__ void load8(const float* p, int lane, float (&x)[8])
{
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p + lane * 4)), b = __ldcs(reinterpret_cast<const float4*>(p + 128 + lane * 4));
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

__device__ __forceinline__ void store8(float* p, int lane, const float (&x)[8])
{
    __stcs(reinterpret_cast<float4*>(p + lane * 4), make_float4(x[0], x[1], x[2], x[3]));
    __stcs(reinterpret_cast<float4*>(p + 128 + lane * 4), make_float4(x[4], x[5], x[6], x[7]));
}

// ---------------------------------------------------------------- blocks on their way

// With 8-bit moments a warp's aligned blocks come through shared memory of its own, copied
// asynchronously two blocks ahead (their records four ahead), so that no register waits for memory:
// the arithmetic needs them.  Measured on GB300 (124M elements, fp16 gradients), before the roots were rounded
// exactly: loads into registers 361 us, one, two, three, four blocks ahead 348, 335, 343, 373.  The exact roots
// bound the step since (362 us), and the depth shows less: with the export 478, 475, 474 and 479.  With 32-bit moments the
// arithmetic is less and plain loads with 24 warps an SM are faster (59M elements: 268 us against
// 288).
template <int GT>
struct Ring {
    static constexpr int kStages = kAhead + 1, kRecords = 2 * kAhead + 1;
    static constexpr int kG = GT == ZERO_FP32 ? 2 : 1;                              // a lane's pieces of g
    static constexpr int kP = kG * 512 + 16, kM = kP + 1024;     // places of p and the moments
    static constexpr int kStage = kM + 2 * kBlockElems;
    static constexpr int kWarp = kStages * kStage + kRecords * 32;
    static constexpr int kBytes = kAdamWarps * kWarp;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void copy4(uint32_t dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ uint32_t shared4(uint32_t at)
{
    uint32_t q;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(q) : "r"(at) : "memory");
    return q;
}

__device__ __forceinline__ uint4 shared16(uint32_t at)
{
    uint4 q;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(at) : "memory");
    return q;
}

__device__ __forceinline__ uint2 shared8(uint32_t at)
{
    uint2 q;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(q.x), "=r"(q.y) : "r"(at) : "memory");
    return q;
}

__device__ __forceinline__ AdamBlock shared_block(uint32_t at)
{
    AdamBlock B;
    reinterpret_cast<uint4*>(&B)[0] = shared16(at);
    reinterpret_cast<uint4*>(&B)[1] = shared16(at + 16);
    return B;
}

// Start the copies of block b into a stage: g, p, m and v one after the other.
template <int GT>
__device__ __forceinline__ void start_block(const AdamParams& P, const AdamBlock& B, int b, int lane, uint32_t stage)
{
    using R = Ring<GT>;
    if (B.vec == kSingly) return;
    if (B.vec == kAligned) {
        const uint32_t own = stage + lane * 16;
        const char* g = static_cast<const char*>(B.g) + lane * 16;
        const char* p = reinterpret_cast<const char*>(B.p) + lane * 16;
#pragma unroll
        for (int i = 0; i < R::kG; ++i) copy16(own + i * 512, g + i * 512);
#pragma unroll
        for (int i = 0; i < 2; ++i) copy16(own + R::kP + i * 512, p + i * 512);
    } else {
        // words; 16-bit gradients that start in the middle of one take 129
        const uint32_t own = stage + lane * 4, off = (uint32_t)(uintptr_t)B.g & 3u;
        const char* g = static_cast<const char*>(B.g) - off + lane * 4;
        const char* p = reinterpret_cast<const char*>(B.p) + lane * 4;
#pragma unroll
        for (int i = 0; i < 4 * R::kG; ++i) copy4(own + i * 128, g + i * 128);
        if (off && lane == 0) copy4(own + 512, g + 512);
#pragma unroll
        for (int i = 0; i < 8; ++i) copy4(own + R::kP + i * 128, p + i * 128);
    }
    const uint32_t moments = stage + R::kM;
    // m by the first half of the warp, v by the second
    const uint32_t half = lane >> 4, k = (lane & 15) * 16;
    const char* m = static_cast<const char*>(half ? P.v : P.m) + (int64_t)b * kBlockElems;
    copy16(moments + half * kBlockElems + k, m + k);
}

// A lane's eight values of one of them.
__device__ __forceinline__ void take_fp32(uint32_t at, int lane, float (&x)[8])
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 q = shared16(at + i * 512 + lane * 16);
        x[4 * i] = __uint_as_float(q.x);
        x[4 * i + 1] = __uint_as_float(q.y);
        x[4 * i + 2] = __uint_as_float(q.z);
        x[4 * i + 3] = __uint_as_float(q.w);
    }
}

template <int GT>
__device__ __forceinline__ void take_grads(const AdamBlock& B, uint32_t at, int lane, float (&x)[8])
{
    if constexpr (GT == ZERO_FP32) {
        take_fp32(at, lane, x);
    } else {
        const bool middle = B.vec == kInner && ((uint32_t)(uintptr_t)B.g & 2u);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint2 q = shared8(at + i * 256 + lane * 8);
            if (middle) {
                const uint32_t last = shared4(at + i * 256 + lane * 8 + 8);
                q = make_uint2(__byte_perm(q.x, q.y, 0x5432u), __byte_perm(q.y, last, 0x5432u));
            }
            widen2<GT>(q.x, x[4 * i], x[4 * i + 1]);
            widen2<GT>(q.y, x[4 * i + 2], x[4 * i + 3]);
        }
    }
}

__device__ __forceinline__ uint2 take_codes(uint32_t at, int lane)
{
    uint2 c;
    c.x = shared4(at + lane * 4);
    c.y = shared4(at + 128 + lane * 4);
    return c;
}

// ---------------------------------------------------------------- 8-bit moments
//
// Codes are handled in pairs, one in each half of a word: code << 6 in 16 bits is the half-precision
// number of half the value in units of the scale (4 of its 5 exponent bits, 4 of its 10 fraction
// bits; subnormals too), so the conversions between fp16 and fp32 do the work.

__device__ __forceinline__ void decode_m2(uint32_t two, F2 scale, float& a, float& b)
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    split(mul(pair(f.x, f.y), scale), a, b);
}

__device__ __forceinline__ uint32_t encode_m2(float a, float b, F2 inv)
{
    float2 f;
    split(mul(pair(a, b), inv), f.x, f.y);
    return __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
}

// scale2 = twice the root's scale.  two: the codes in the low bytes of the halves.
__device__ __forceinline__ void decode_root2(uint32_t two, F2 scale2, float& a, float& b)
{
    const uint32_t w = two << 6;
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    split(mul(pair(f.x, f.y), scale2), a, b);
}

// The power of two whose last place is x's fifth: x plus it, minus it, is x to four fraction bits (below
// 2^-14, fp16's and the code's smallest normal number, to a multiple of 2^-18), to nearest, ties to even.
__device__ __forceinline__ float rounder(float x)
{
    return __uint_as_float(max(__float_as_uint(x) & 0x7F800000u, 113u << 23) + (19u << 23));
}

// inv_half = half of the scale's inverse.  A root above 0 is at least code 1.
__device__ __forceinline__ uint32_t encode_root2(float a, float b, F2 inv_half)
{
    float x, y;
    split(mul(pair(a, b), inv_half), x, y);
    if (a > 0.0f) x = fmaxf(x, 0x1p-18f);
    if (b > 0.0f) y = fmaxf(y, 0x1p-18f);
    const float rx = rounder(x), ry = rounder(y);
    x = __fsub_rn(__fadd_rn(x, rx), rx);
    y = __fsub_rn(__fadd_rn(y, ry), ry);
    uint32_t h;
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(y), "f"(x));
    return (h >> 6) & 0x00FF00FFu;
}

// Whether one of four code bytes is 255, the mark of a root that is not finite.
__device__ __forceinline__ bool marked(uint32_t c) { return ((c & 0x7F7F7F7Fu) + 0x01010101u) & c & 0x80808080u; }

__device__ __forceinline__ void mark_roots(uint32_t lo, uint32_t hi, float (&r)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if ((((j < 4 ? lo : hi) >> (8 * (j & 3))) & 0xFFu) == 0xFFu) r[j] = __uint_as_float(0x7FC00000u);
}

// Exponent field of the warp's largest finite magnitude; a value that is not finite becomes not a number
// (an infinite m would saturate to a finite code).
__device__ __noinline__ uint32_t top_field_of_finite(float* x)
{
    uint32_t top = 0;
    for (int j = 0; j < 8; ++j) {
        if (nonfinite(x[j])) x[j] = __uint_as_float(0x7FC00000u);
        else top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
    }
    return __reduce_max_sync(0xFFFFFFFFu, top) >> 23;
}

// The pair (2 i, 2 i + 1) of a lane's eight code bytes, one in each half; and back.
__device__ __forceinline__ uint32_t code_pair(uint2 c, int i)
{
    return __byte_perm(i < 2 ? c.x : c.y, 0u, (i & 1) ? 0x4342u : 0x4140u);
}

__device__ __forceinline__ float reciprocal_approx(float d)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    return r;
}

__device__ __forceinline__ float root_approx(float v)
{
    float r;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// ---------------------------------------------------------------- kernels

// fp32(1 / loss scale), as the sharded step forms it.
__device__ __forceinline__ float unscale(const volatile DevState* plan)
{
    return __double2float_rn(__ddiv_rn(1.0, plan->scale));
}

template <int BITS, int GT, int DT>
__global__ void __launch_bounds__(kAdamThreads, BITS == 8 ? kAdamPerSm8 : kAdamPerSm32) adamw_kernel(const __grid_constant__ AdamParams P)
{
    after_earlier_work();
    __shared__ float sk_shared[4];
    __shared__ bool skip;
    using R = Ring<GT>;
    constexpr bool kRing = BITS == 8;
    extern __shared__ __align__(16) unsigned char ring[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int stride = gridDim.x * kAdamWarps;
    const uint32_t mine = (uint32_t)__cvta_generic_to_shared(ring) + warp * R::kWarp;
    const uint32_t records = mine + R::kStages * R::kStage;
    int b = blockIdx.x * kAdamWarps + warp;
    auto start_record = [&](int k, int at) {
        if (lane < 2 && at < P.n_blocks) copy16(records + (k % R::kRecords) * 32 + lane * 16, reinterpret_cast<const char*>(P.blocks + at) + lane * 16);
    };
    uint32_t scales0 = 0, scales1 = 0;           // of this block and the next
    AdamBlock next = {};
    if constexpr (kRing) {
        if (b < P.n_blocks) scales0 = P.scales[b];
        if (b + stride < P.n_blocks) scales1 = P.scales[b + stride];
        // the first blocks, and the records of as many after them
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (b + k * stride < P.n_blocks) start_block<GT>(P, block_at(P, b + k * stride), b + k * stride, lane, mine + k * R::kStage);
            start_record(k, b + k * stride);
            start_record(k + kAhead, b + (k + kAhead) * stride);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    } else {
        if (b < P.n_blocks) next = block_at(P, b);
    }
    // the constants of this step, while the first loads are on their way: two lanes raise the betas
    // to the step's power
    if (threadIdx.x < 32) {
        const volatile AdamState* st = P.st;
        const int64_t t = st->t + 1;
        const double bc = 1.0 - pow_int(lane == 0 ? P.beta1 : P.beta2, t);
        if (lane == 0) {
            sk_shared[0] = __double2float_rn(__ddiv_rn(P.lr, bc));
            const volatile DevState* plan = P.plan;
            float coef = 1.0f, inv = P.inv;
            bool s = false;
            if (plan) {
                s = (plan->flag | plan->error) != 0;
                inv = unscale(plan);
            } else if (P.checked) {
                s = st->flag != 0;
            }
            if (P.max_norm > 0.0) {
                const double norm2 = plan ? plan->norm2 : st->norm2;
                const double c = __ddiv_rn(P.max_norm, __dadd_rn(__dsqrt_rn(norm2), 1e-6));
                coef = __double2float_rn(c > 1.0 ? 1.0 : c);
            }
            // the gradient is multiplied by 1 / loss scale, then by the clipping coefficient; where
            // one of them is 1 that is one product
            const bool one = inv == 1.0f || coef == 1.0f;
            sk_shared[2] = one ? inv * coef : inv;
            sk_shared[3] = one ? 1.0f : coef;
            skip = s;
        } else if (lane == 1) {
            sk_shared[1] = __double2float_rn(__ddiv_rn(1.0, __dsqrt_rn(bc)));
        }
    }
    __syncthreads();
    const F2 minus_step = both(-sk_shared[0]), inv_bc2s = both(sk_shared[1]), inv = both(sk_shared[2]), coef = both(sk_shared[3]);
    const bool twice = sk_shared[3] != 1.0f;

    if (!skip) {
        for (int k = 0; b < P.n_blocks; ++k, b += stride) {
            const int block = b;
            const int64_t s0 = (int64_t)block * kBlockElems;              // in the moments
            AdamBlock B;
            uint32_t scales = 0;
            if constexpr (kRing) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
                __syncwarp();
                B = shared_block(records + (k % R::kRecords) * 32);
                if (b + kAhead * stride < P.n_blocks)
                    start_block<GT>(P, shared_block(records + ((k + kAhead) % R::kRecords) * 32), b + kAhead * stride, lane,
                                    mine + ((k + kAhead) % R::kStages) * R::kStage);
                start_record(k + 2 * kAhead, b + 2 * kAhead * stride);
                asm volatile("cp.async.commit_group;" ::: "memory");
                scales = scales0;
                scales0 = scales1;
                if (b + 2 * stride < P.n_blocks) scales1 = P.scales[b + 2 * stride];
            } else {
                B = next;
                if (b + stride < P.n_blocks) next = block_at(P, b + stride);
            }
            // with the ring, inner blocks are read as aligned ones are
            const bool vec = kRing ? B.vec != kSingly : B.vec == kAligned;
            float g[8], p[8], m[8], v[8];
            if (vec) {
                if constexpr (!kRing) {
                    load_grads<GT>(B, lane, g);
                    load8(B.p, lane, p);
                    load8(static_cast<const float*>(P.m) + s0, lane, m);
                    load8(static_cast<const float*>(P.v) + s0, lane, v);
                } else {
                    const uint32_t stage = mine + (k % R::kStages) * R::kStage, moments = stage + R::kM;
                    take_grads<GT>(B, stage, lane, g);
                    take_fp32(stage + R::kP, lane, p);
                    const F2 ms = both(power_field(scales & 0xFFu)), rs = both(power_field(scales >> 8) * 2.0f);
                    const uint2 mc = take_codes(moments, lane), vc = take_codes(moments + kBlockElems, lane);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        decode_m2((i < 2 ? mc.x : mc.y) >> (16 * (i & 1)), ms, m[2 * i], m[2 * i + 1]);
                        decode_root2(code_pair(vc, i), rs, v[2 * i], v[2 * i + 1]);
                    }
                    if (marked(vc.x) || marked(vc.y)) mark_roots(vc.x, vc.y, v);
                }
            } else {
                const float* bp = B.p + lane;
                const char* bg = static_cast<const char*>(B.g) + lane * (GT == ZERO_FP32 ? 4 : 2);
                if (B.n == kBlockElems) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        g[j] = load_grad1<GT>(bg, j * 32);
                        p[j] = bp[j * 32];
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const bool in = j * 32 + lane < B.n;
                        g[j] = in ? load_grad1<GT>(bg, j * 32) : 0.0f;
                        p[j] = in ? bp[j * 32] : 0.0f;
                    }
                }
                if constexpr (BITS == 32) {
                    const float* mp = static_cast<const float*>(P.m) + s0 + lane;
                    const float* vp = static_cast<const float*>(P.v) + s0 + lane;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        m[j] = mp[j * 32];
                        v[j] = vp[j * 32];
                    }
                } else {
                    const F2 ms = both(power_field(scales & 0xFFu)), rs = both(power_field(scales >> 8) * 2.0f);
                    const uint8_t* mp = static_cast<const uint8_t*>(P.m) + s0 + lane;
                    const uint8_t* vp = static_cast<const uint8_t*>(P.v) + s0 + lane;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        decode_m2(mp[i * 64] | ((uint32_t)mp[i * 64 + 32] << 8), ms, m[2 * i], m[2 * i + 1]);
                        const uint32_t c = vp[i * 64] | ((uint32_t)vp[i * 64 + 32] << 16);
                        decode_root2(c, rs, v[2 * i], v[2 * i + 1]);
                        if (marked(c)) {
                            if ((c & 0xFFu) == 0xFFu) v[2 * i] = __uint_as_float(0x7FC00000u);
                            if (c >> 16 == 0xFFu) v[2 * i + 1] = __uint_as_float(0x7FC00000u);
                        }
                    }
                }
            }
            float root[8];
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                F2 gu = mul(pair(g[i], g[i + 1]), inv);
                if (twice) gu = mul(gu, coef);
                F2 v2 = pair(v[i], v[i + 1]);
                if constexpr (BITS == 8) v2 = mul(v2, v2);
                // every product and sum rounded by itself: an 8-bit moment is a small whole number of
                // units, so that exact ties of its next value are common and a last place decides them
                const F2 m2 = add_apart(mul(P.k[0], pair(m[i], m[i + 1])), mul(P.k[1], gu), P.one);
                v2 = add_apart(mul(P.k[2], v2), mul(P.k[3], mul(gu, gu)), P.one);
                split(m2, m[i], m[i + 1]);
                split(v2, v[i], v[i + 1]);
                // a root that is stored is rounded exactly, as its code has to follow from the values alone;
                // else it is within 2 units in the last place, as the quotient is, on a step that is a small
                // part of the parameter it is added to
                root[i] = BITS == 8 ? __fsqrt_rn(v[i]) : root_approx(v[i]);
                root[i + 1] = BITS == 8 ? __fsqrt_rn(v[i + 1]) : root_approx(v[i + 1]);
                float d0, d1;
                split(add_apart(mul(pair(root[i], root[i + 1]), inv_bc2s), P.k[4], P.one), d0, d1);
                F2 p2 = pair(p[i], p[i + 1]);
                p2 = add_apart(mul(P.k[5], p2), p2, P.one);
                p2 = add_apart(mul(minus_step, mul(m2, pair(reciprocal_approx(d0), reciprocal_approx(d1)))), p2, P.one);
                split(p2, p[i], p[i + 1]);
            }
            if (kRing && B.vec == kInner) {
                // through the stage: four in a row there, 32 lanes' neighbours to memory
                const uint32_t stage = mine + (k % R::kStages) * R::kStage;
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(stage + R::kP + i * 512 + lane * 16), "f"(p[4 * i]),
                                 "f"(p[4 * i + 1]), "f"(p[4 * i + 2]), "f"(p[4 * i + 3])
                                 : "memory");
                    if (B.p16)
                        asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(stage + i * 256 + lane * 8),
                                     "r"(narrow2<DT>(p[4 * i], p[4 * i + 1])), "r"(narrow2<DT>(p[4 * i + 2], p[4 * i + 3]))
                                     : "memory");
                }
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j) B.p[j * 32 + lane] = __uint_as_float(shared4(stage + R::kP + j * 128 + lane * 4));
                if (B.p16) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        uint16_t h;
                        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(stage + j * 64 + lane * 2) : "memory");
                        B.p16[j * 32 + lane] = h;
                    }
                }
            } else if (vec) {
                store8(B.p, lane, p);
                if (B.p16) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        __stcs(reinterpret_cast<uint2*>(B.p16 + i * 128 + lane * 4),
                               make_uint2(narrow2<DT>(p[4 * i], p[4 * i + 1]), narrow2<DT>(p[4 * i + 2], p[4 * i + 3])));
                }
            } else if (B.n == kBlockElems) {
#pragma unroll
                for (int j = 0; j < 8; ++j) B.p[j * 32 + lane] = p[j];
                if (B.p16) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) B.p16[j * 32 + lane] = narrow1<DT>(p[j]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int e = j * 32 + lane;
                    if (e < B.n) {
                        B.p[e] = p[j];
                        if (B.p16) B.p16[e] = narrow1<DT>(p[j]);
                    } else {
                        m[j] = v[j] = root[j] = 0.0f;      // the moments' padding stays zero
                    }
                }
            }
            if constexpr (BITS == 32) {
                float* mp = static_cast<float*>(P.m) + s0;
                float* vp = static_cast<float*>(P.v) + s0;
                if (vec) {
                    store8(mp, lane, m);
                    store8(vp, lane, v);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        mp[j * 32 + lane] = m[j];
                        vp[j * 32 + lane] = v[j];
                    }
                }
            } else {
                // the block's largest magnitudes; m is finite where the root is
                uint32_t top_r = 0;
                float top_m = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    top_r = max(top_r, __float_as_uint(root[j]) & 0x7FFFFFFFu);
                    top_m = fmaxf(top_m, fabsf(m[j]));
                }
                top_r = __reduce_max_sync(0xFFFFFFFFu, top_r);
                uint32_t er = top_r >> 23, fm = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top_m)) >> 23;
                const bool finite = er != 0xFFu;
                if (!finite) {
                    er = top_field_of_finite(root);
                    fm = top_field_of_finite(m);
                }
                const uint32_t em = fm > 8u ? fm - 7u : 1u;
                const F2 mi = both(power_field(254u - em)), ri = both(power_field(254u - er) * 0.5f);
                uint32_t mc[4], rc[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mc[i] = encode_m2(m[2 * i], m[2 * i + 1], mi);
                    rc[i] = encode_root2(root[2 * i], root[2 * i + 1], ri);
                }
                if (!finite) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (nonfinite(root[2 * i])) rc[i] = (rc[i] & 0xFFFF0000u) | 0xFFu;
                        if (nonfinite(root[2 * i + 1])) rc[i] = (rc[i] & 0x0000FFFFu) | 0x00FF0000u;
                    }
                }
                uint8_t* mp = static_cast<uint8_t*>(P.m) + s0;
                uint8_t* vp = static_cast<uint8_t*>(P.v) + s0;
                if (vec) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        __stcs(reinterpret_cast<uint32_t*>(mp + i * 128 + lane * 4), mc[2 * i] | (mc[2 * i + 1] << 16));
                        __stcs(reinterpret_cast<uint32_t*>(vp + i * 128 + lane * 4), __byte_perm(rc[2 * i], rc[2 * i + 1], 0x6420u));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        mp[i * 64 + lane] = (uint8_t)mc[i];
                        mp[i * 64 + 32 + lane] = (uint8_t)(mc[i] >> 8);
                        vp[i * 64 + lane] = (uint8_t)rc[i];
                        vp[i * 64 + 32 + lane] = (uint8_t)(rc[i] >> 16);
                    }
                }
                if (lane == 0) P.scales[block] = (uint16_t)(em | (er << 8));
            }
        }
    }
    if constexpr (kRing) asm volatile("cp.async.wait_all;" ::: "memory");
    // the last block to finish closes the step: every block has read t by then (and nothing else of
    // theirs is read here, so that no store has to be waited for)
    __syncthreads();
    if (threadIdx.x == 0) {
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
// sum is fixed: lanes, then warps, then blocks in order.  JOINED: both go to a sharded step's state, to what its
// own passes have found.
template <int GT, bool JOINED>
__global__ void __launch_bounds__(kAdamThreads) adamw_norm_kernel(const __grid_constant__ AdamParams P)
{
    after_earlier_work();
    __shared__ double warp_sum[kAdamWarps];
    __shared__ bool last;
    const int lane = threadIdx.x & 31;
    // error-free sums (TwoSum, Knuth) of pairs of squares; a value that is not finite makes them so
    F2 hi = both(0.0f), lo = both(0.0f);
    const F2 inv = both(JOINED ? unscale(P.plan) : P.inv), minus = both(-1.0f);
    const int stride = gridDim.x * kAdamWarps;
    int b = blockIdx.x * kAdamWarps + (threadIdx.x >> 5);
    AdamBlock next = {};
    if (b < P.n_blocks) next = block_at(P, b);
    while (b < P.n_blocks) {
        const AdamBlock B = next;
        float g[8];
        load_grads<GT>(B, lane, g);
        b += stride;
        if (b < P.n_blocks) next = block_at(P, b);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const F2 x = mul(pair(g[j], g[j + 1]), inv), p = mul(x, x);
            const F2 s = add_apart(p, hi, P.one);
            const F2 bp = fma(hi, minus, s), ap = fma(bp, minus, s);
            lo = add(lo, add(fma(ap, minus, hi), add_apart(p, fma(bp, minus, both(0.0f)), P.one)));
            hi = s;
        }
    }
    float h0, h1, l0, l1;
    split(hi, h0, h1);
    split(lo, l0, l1);
    const double mine = ((double)h0 + (double)h1) + ((double)l0 + (double)l1);
    const double s = block_sum_fixed<kAdamThreads>(mine, warp_sum);
    if (threadIdx.x == 0) {
        P.partials[blockIdx.x] = s;
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
        if constexpr (JOINED) {
            volatile DevState* plan = P.plan;
            plan->norm2 = plan->norm2 + sum;
            if (!isfinite(sum)) plan->flag = 1u;
        } else {
            st->norm2 = sum;
            st->flag = isfinite(sum) ? 0u : 1u;
        }
        st->norm_tickets = 0;
    }
}

// The table of blocks from the table of tensors.
__global__ void __launch_bounds__(kAdamThreads) adamw_table_kernel(const AdamTensor* tensors, int64_t n, int grad_bytes,
                                                                   AdamBlock* blocks)
{
    after_earlier_work();
    for (int64_t i = blockIdx.x; i < n; i += gridDim.x) {
        const AdamTensor T = tensors[i];
        const int64_t count = (T.n + kBlockElems - 1) / kBlockElems;
        for (int64_t k = threadIdx.x; k < count; k += kAdamThreads) {
            const int64_t e = k * kBlockElems;
            AdamBlock B;
            B.p = T.p + e;
            B.p16 = T.p16 ? T.p16 + e : nullptr;
            B.g = static_cast<const char*>(T.g) + e * grad_bytes;
            B.n = (int32_t)min((int64_t)kBlockElems, T.n - e);
            B.vec = B.n < kBlockElems ? kSingly : T.vec ? kAligned : k > 0 && k + 1 < count ? kInner : kSingly;
            blocks[T.first + k] = B;
        }
    }
}

// The 8-bit moments as the values that they stand for; bf16 holds each of them exactly.
__global__ void __launch_bounds__(kAdamThreads) adamw_export_kernel(const uint8_t* m, const uint8_t* v,
                                                                    const uint16_t* scales, uint16_t* m_out,
                                                                    uint16_t* root_out, int n_blocks)
{
    after_earlier_work();
    const int lane = threadIdx.x & 31, stride = gridDim.x * kAdamWarps;
    for (int b = blockIdx.x * kAdamWarps + (threadIdx.x >> 5); b < n_blocks; b += stride) {
        const int64_t at = (int64_t)b * kBlockElems + lane * 8;
        const uint2 mc = __ldcs(reinterpret_cast<const uint2*>(m + at));
        const uint2 vc = __ldcs(reinterpret_cast<const uint2*>(v + at));
        const uint32_t e = scales[b];
        const F2 ms = both(power_field(e & 0xFFu)), rs = both(power_field(e >> 8) * 2.0f);
        float x[8], r[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            decode_m2((i < 2 ? mc.x : mc.y) >> (16 * (i & 1)), ms, x[2 * i], x[2 * i + 1]);
            decode_root2(code_pair(vc, i), rs, r[2 * i], r[2 * i + 1]);
        }
        if (marked(vc.x) || marked(vc.y)) mark_roots(vc.x, vc.y, r);
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
    // the sharded step (zero_plan::step_no) that zero_adamw_check, zero_adamw_step_with joined last
    int64_t checked_in = 0, stepped_in = 0;
};

namespace zero {
namespace {

// Workspace: the state's slot, the tensors, the blocks, the norm pass's slots.
constexpr int64_t kAdamStateBytes = 256;
inline int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }
int64_t tensors_at() { return kAdamStateBytes; }
int64_t blocks_at(const zero_adamw* h) { return tensors_at() + up16((int64_t)sizeof(AdamTensor) * (int64_t)h->sizes.size()); }
int64_t slots_at(const zero_adamw* h) { return blocks_at(h) + (int64_t)sizeof(AdamBlock) * h->n_blocks; }
int64_t adam_workspace(const zero_adamw* h) { return slots_at(h) + 8 * kAdamNormSlots; }

// A persistent grid: as many blocks as fit the GPU at once, or as the work needs.
template <auto KERNEL, int SHARED = 0>
int adam_grid(const zero_adamw* h)
{
    if constexpr (SHARED > 0) allow_shared<KERNEL>(SHARED);      // a refusal shows at the launch
    static const int per_sm = [] {
        int n = 0;
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, KERNEL, kAdamThreads, SHARED) == cudaSuccess ? std::max(1, n) : 1;
    }();
    const int64_t cap = (int64_t)std::max(1, device_sms(h->device)) * per_sm;
    const int64_t need = (h->n_blocks + kAdamWarps - 1) / kAdamWarps;
    return (int)std::max<int64_t>(1, std::min({cap, need, (int64_t)kAdamNormSlots}));
}

template <int BITS, int GT>
void launch_adamw(const zero_adamw* h, const AdamParams& P, cudaStream_t s)
{
    constexpr int kShared = BITS == 8 ? Ring<GT>::kBytes : 0;
    if (h->dtype16 == ZERO_BF16)
        launch_after(adamw_kernel<BITS, GT, ZERO_BF16>, adam_grid<adamw_kernel<BITS, GT, ZERO_BF16>, kShared>(h), kAdamThreads, kShared, s, P);
    else
        launch_after(adamw_kernel<BITS, GT, ZERO_FP16>, adam_grid<adamw_kernel<BITS, GT, ZERO_FP16>, kShared>(h), kAdamThreads, kShared, s, P);
}

template <int BITS>
void launch_adamw(const zero_adamw* h, const AdamParams& P, cudaStream_t s)
{
    if (h->grad_type == ZERO_BF16) launch_adamw<BITS, ZERO_BF16>(h, P, s);
    else if (h->grad_type == ZERO_FP16) launch_adamw<BITS, ZERO_FP16>(h, P, s);
    else launch_adamw<BITS, ZERO_FP32>(h, P, s);
}

template <int GT, bool JOINED>
void launch_norm(const zero_adamw* h, const AdamParams& P, cudaStream_t s)
{
    launch_after(adamw_norm_kernel<GT, JOINED>, adam_grid<adamw_norm_kernel<GT, JOINED>>(h), kAdamThreads, 0, s, P);
}

template <bool JOINED>
void launch_norm(const zero_adamw* h, const AdamParams& P, cudaStream_t s)
{
    if (h->grad_type == ZERO_BF16) launch_norm<ZERO_BF16, JOINED>(h, P, s);
    else if (h->grad_type == ZERO_FP16) launch_norm<ZERO_FP16, JOINED>(h, P, s);
    else launch_norm<ZERO_FP32, JOINED>(h, P, s);
}

F2 twice(float x)
{
    uint32_t w;
    std::memcpy(&w, &x, 4);
    return F2{((unsigned long long)w << 32) | w};
}

// What every pass over the bound tensors needs.
AdamParams adam_params(const zero_adamw* h)
{
    char* ws = static_cast<char*>(h->workspace);
    AdamParams P;
    std::memset(&P, 0, sizeof(P));
    P.blocks = reinterpret_cast<const AdamBlock*>(ws + blocks_at(h));
    P.m = h->m;
    P.v = h->v;
    P.scales = static_cast<uint16_t*>(h->scales);
    P.st = reinterpret_cast<AdamState*>(ws);
    P.partials = reinterpret_cast<double*>(ws + slots_at(h));
    P.n_blocks = (int32_t)h->n_blocks;
    P.one = twice(1.0f);
    P.inv = 1.0f;
    return P;
}

zero_status_t check_hyper(const zero_hyper_t* hyper, const char* who)
{
    const std::string w = std::string(who) + ": ";
    if (!(hyper->beta1 >= 0.0 && hyper->beta1 < 1.0) || !(hyper->beta2 >= 0.0 && hyper->beta2 < 1.0))
        return fail(ZERO_EINVAL, w + "betas must be in [0, 1)");
    if (!(hyper->eps >= 0.0) || !(hyper->max_grad_norm >= 0.0) || !std::isfinite(hyper->lr) ||
        !std::isfinite(hyper->weight_decay))
        return fail(ZERO_EINVAL, w + "bad hyperparameter");
    if (hyper->flags & ~(int64_t)ZERO_REPORT_GRAD_NORM) return fail(ZERO_EINVAL, w + "unknown flag");
    return ZERO_OK;
}

// The step's constants into P.
void set_hyper(AdamParams& P, const zero_hyper_t& hyper, double loss_scale)
{
    float c[9];
    step_constants(hyper, 1, loss_scale, 1, c);
    // eps: the smallest normal number at least, so that its reciprocal is finite
    if (c[4] > 0.0f && c[4] < 0x1p-126f) c[4] = 0x1p-126f;
    c[5] = -c[5];
    for (int i = 0; i < 6; ++i) P.k[i] = twice(c[i]);
    P.inv = c[8];
    P.lr = hyper.lr;
    P.beta1 = hyper.beta1;
    P.beta2 = hyper.beta2;
    P.max_norm = hyper.max_grad_norm;
}

void launch_adamw(const zero_adamw* h, const AdamParams& P, cudaStream_t s)
{
    if (h->bits == 8) launch_adamw<8>(h, P, s);
    else launch_adamw<32>(h, P, s);
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

// The plan whose step h joins: bound, on h's device.
zero_status_t plan_ready(const zero_adamw* h, const zero_plan* plan, const char* who)
{
    if (!h || !plan) return fail(ZERO_EINVAL, std::string(who) + ": NULL argument");
    const zero_status_t st = adam_ready(h, who);
    if (st != ZERO_OK) return st;
    if (!plan->workspace) return fail(ZERO_ESTATE, std::string(who) + ": no rank of the plan is bound");
    if (plan->device != h->device) return fail(ZERO_EINVAL, std::string(who) + ": the plan lives on another device");
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
    std::vector<unsigned char> image((size_t)(blocks_at(h)), 0);
    AdamTensor* T = reinterpret_cast<AdamTensor*>(image.data() + tensors_at());
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
        block += (elems + kBlockElems - 1) / kBlockElems;
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
    if (e == cudaSuccess && h->n_blocks > 0) {
        char* ws = static_cast<char*>(workspace);
        launch_after(adamw_table_kernel, (unsigned)std::min<int64_t>((int64_t)n, 4096), kAdamThreads, 0, s, reinterpret_cast<const AdamTensor*>(ws + tensors_at()), (int64_t)n, (int)gsize,
            reinterpret_cast<AdamBlock*>(ws + blocks_at(h)));
        e = cudaGetLastError();
    }
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e, "zero_adamw_bind: the workspace's tables");
    h->m = m;
    h->v = v;
    h->scales = scales;
    h->workspace = workspace;
    h->checked_in = 0;                           // other gradients than a check saw
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
    zero_status_t st = check_hyper(hyper, "zero_adamw_step");
    if (st != ZERO_OK) return st;
    if (!(loss_scale > 0.0) || !std::isfinite(loss_scale))
        return fail(ZERO_EINVAL, "zero_adamw_step: loss_scale must be positive");
    st = adam_ready(h, "zero_adamw_step");
    if (st != ZERO_OK) return st;
    AdamParams P = adam_params(h);
    set_hyper(P, *hyper, loss_scale);
    P.checked = hyper->max_grad_norm > 0.0 || (hyper->flags & ZERO_REPORT_GRAD_NORM);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (P.checked) launch_norm<false>(h, P, s);
    launch_adamw(h, P, s);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? ZERO_OK : cuda_fail(e, "zero_adamw_step: launch");
}
catch (...) {
    return exception_status("zero_adamw_step");
}

zero_status_t zero_adamw_check(zero_adamw_t* h, zero_plan_t* plan, void* stream)
try {
    const zero_status_t st = plan_ready(h, plan, "zero_adamw_check");
    if (st != ZERO_OK) return st;
    if (h->checked_in == plan->step_no) return fail(ZERO_ESTATE, "zero_adamw_check: already part of this step");
    if (plan->in_step && (plan->offload || plan->step_hyper.max_grad_norm > 0.0))
        return fail(ZERO_ESTATE, "zero_adamw_check: must precede the first bucket/unit of a step that clips or is offloaded");
    if (plan->moved_in == plan->step_no) return fail(ZERO_ESTATE, "zero_adamw_check: a part of this step, which it could not leave out, is enqueued");
    AdamParams P = adam_params(h);
    P.plan = reinterpret_cast<DevState*>(plan->workspace);
    launch_norm<true>(h, P, static_cast<cudaStream_t>(stream));
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "zero_adamw_check: launch");
    h->checked_in = plan->step_no;
    return ZERO_OK;
}
catch (...) {
    return exception_status("zero_adamw_check");
}

zero_status_t zero_adamw_step_with(zero_adamw_t* h, zero_plan_t* plan, const zero_hyper_t* hyper, void* stream)
try {
    if (!hyper) return fail(ZERO_EINVAL, "zero_adamw_step_with: NULL argument");
    zero_status_t st = check_hyper(hyper, "zero_adamw_step_with");
    if (st == ZERO_OK) st = plan_ready(h, plan, "zero_adamw_step_with");
    if (st != ZERO_OK) return st;
    if (h->checked_in != plan->step_no) return fail(ZERO_ESTATE, "zero_adamw_step_with: needs zero_adamw_check in the same step");
    if (h->stepped_in == plan->step_no) return fail(ZERO_ESTATE, "zero_adamw_step_with: already part of this step");
    bool all = plan->in_step;
    for (int64_t b = 0; b < plan->n_buckets && all; ++b) all = plan->covered[(size_t)b] != 0;
    if (!all) return fail(ZERO_ESTATE, "zero_adamw_step_with: follows the step of every bucket/unit, before the step's finish");
    if (hyper->max_grad_norm != plan->step_hyper.max_grad_norm)
        return fail(ZERO_EINVAL, "zero_adamw_step_with: one step has one max_grad_norm");
    AdamParams P = adam_params(h);
    set_hyper(P, *hyper, 1.0);
    P.plan = reinterpret_cast<DevState*>(plan->workspace);
    plan->moved_in = plan->step_no;
    launch_adamw(h, P, static_cast<cudaStream_t>(stream));
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "zero_adamw_step_with: launch");
    h->stepped_in = plan->step_no;
    return ZERO_OK;
}
catch (...) {
    return exception_status("zero_adamw_step_with");
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
    launch_after(adamw_export_kernel, adam_grid<adamw_export_kernel>(h), kAdamThreads, 0, static_cast<cudaStream_t>(stream), static_cast<const uint8_t*>(h->m), static_cast<const uint8_t*>(h->v), static_cast<const uint16_t*>(h->scales),
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
